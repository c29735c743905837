"""The dense products' kernels that only large or particular sizes take, against
plain 64-bit forms, within the bounds dense_ref derives."""

import pytest
import torch

import dense_ref
import test_gpu_dense
from dense_ref import U16, acc_err, close, d64
from gpu_util import DEV, say
from moe_expert_layer_r3_amd import ops
from moe_expert_layer_r3_amd.dense import LinearPlan
from test_gpu_dense import normal

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def on_gpu():
    dense_ref.REF[0] = DEV
    yield
    dense_ref.REF[0] = "cpu"


@pytest.mark.parametrize("T, K, N", [(8200, 4104, 40), (4700, 7176, 256)])
def test_large_data_gradient_with_and_without_the_weights(T, K, N):
    """dx of 64 MB and more is stored past the caches where dW follows: the same
    bits as alone, and nothing behind its last row."""
    say(f"dx T={T} K={K} N={N}")
    W, x, dy = normal((N, K), 1, 0.1), normal((T, K), 2), normal((T, N), 3)
    p = LinearPlan(T, K, N, train=True, device=DEV)
    both = p.backward(dy, x, W)[0].clone()
    buf = torch.full((T + 1, K), 5.0, dtype=BF, device=DEV)
    ptr = lambda t: None if t is None else t.data_ptr()
    for dW in (None, p.dW):
        buf.fill_(5)
        ops.launch("moe_linear_backward", x.device, ptr(dy), 0, None, ptr(x), K, ptr(W), K, None, T, N, K, 0, ptr(buf),
                   ptr(dW), None, ptr(p.ws), p.ws_bytes)
        assert torch.equal(buf[:T], both) and (buf[T] == 5).all()
    D, Wd = d64(dy), d64(W)
    ref = D @ Wd
    e = acc_err(N, D, Wd)
    close(both, ref, e + U16 * (ref.abs() + e), "dx")
    X = d64(x)
    ref = D.t() @ X
    e = acc_err(T, D.t(), X)
    close(p.dW, ref, e + U16 * (ref.abs() + e), "dW")


# ---------------------------------------------------------------- every kernel's every form
# sizes with remainders along M, N and K whose products take the named kernel, K whole
# or in pieces that a second launch adds up

SIZES = [("small", False, 129, 8, 8), ("small", True, 129, 8, 2056), ("tiles", False, 1500, 4104, 136),
         ("tiles", True, 7001, 264, 1544), ("half", False, 3081, 1288, 520), ("half", True, 1237, 776, 3080),
         ("wide", False, 2049, 4104, 776), ("wide", True, 12003, 136, 3080)]


def takes(kernel, pieces, M, N, K, product):
    name, n = ops.dense_kernel(M, N, K, product)
    assert (name, n > 0) == (kernel, pieces), (name, n)


@pytest.mark.parametrize("kernel, pieces, M, N, K", SIZES)
@pytest.mark.parametrize("form", ["plain", "vec", "odd"])
def test_forward_forms(kernel, pieces, M, N, K, form):
    """plain: bf16 of sum, bias and residual; vec: the same with an activation, its
    argument saved, four columns at a time; odd: fp32 out of an odd number of columns."""
    N = N - 3 if form == "odd" else N
    takes(kernel, pieces, M, N, K, "forward")
    name = "none" if form == "plain" else "gelu"
    if form != "odd":
        test_gpu_dense.check_linear(M, K, N, name, False, True, True, form == "vec", pad=8)
    else:
        test_gpu_dense.check_linear(M, K, N, name, True, True, True, False)
        test_gpu_dense.check_linear(M, K, N, "none", True, False, False, False, pad=8)


@pytest.mark.parametrize("kernel, pieces, M, N, K", SIZES)
def test_gradient_forms(kernel, pieces, M, N, K):
    """dx [M, N] = dy [M, K] W [K, N] and dW [M, N] = dy [K, M]^T x [K, N], each alone."""
    takes(kernel, pieces, M, N, K, "gradient")
    say(f"gradients {kernel} pieces={pieces} M={M} N={N} K={K}")
    ptr = lambda t: None if t is None else t.data_ptr()

    def run(T, cols, sums, dx, dW, dy, x, W, add):
        n = ops.workspace_bytes("moe_linear_backward_workspace", T, sums, cols)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        ops.launch("moe_linear_backward", dy.device, ptr(dy), 0, None, ptr(x), 0 if x is None else x.stride(0), ptr(W),
                   0 if W is None else W.stride(0), ptr(add), T, sums, cols, 0, ptr(dx), ptr(dW), None, ptr(ws), ws.numel())

    dy, W, add = normal((M, K), 1), normal((K, N), 2, 0.1, pad=8), normal((M, N), 3)
    out = torch.full((M + 1, N), 5.0, dtype=BF, device=DEV)
    run(M, N, K, out, None, dy, None, W, add)
    D, Wd = d64(dy), d64(W)
    ref = D @ Wd + d64(add)
    e = acc_err(K, D, Wd) + (K + 8) * 2.0 ** -24 * d64(add).abs()
    close(out[:M], ref, e + U16 * (ref.abs() + e) + 1e-30, "dx")
    assert (out[M] == 5).all()

    # (M odd: dy is copied to rows of whole 16 bytes first)
    dy, x = normal((K, M), 4), normal((K, N), 5, pad=8)
    out.fill_(5)
    run(K, N, M, None, out, dy, x, None, None)
    D, X = d64(dy).t(), d64(x)
    ref = D @ X
    e = acc_err(K, D, X)
    close(out[:M], ref, e + U16 * (ref.abs() + e) + 1e-30, "dW")
    assert (out[M] == 5).all()


@pytest.mark.parametrize("kernel, pieces, T, f, d", [
    ("small", False, 129, 8, 8), ("small", True, 129, 8, 2056), ("tiles", False, 1500, 2056, 136),
    ("tiles", True, 1803, 648, 2056), ("half", False, 3081, 648, 520), ("half", True, 1237, 392, 3080),
    ("wide", False, 2049, 2056, 776), ("wide", True, 12003, 72, 3080)])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_forms(kernel, pieces, T, f, d, name):
    """[G, U] of moe_gated_ffn, saved in bf16, with biases and without."""
    takes(kernel, pieces, T, 2 * f, d, "gated")
    test_gpu_dense.check_ffn(T, d, f, name, "bf16", name == "silu", True, pad=8)


@pytest.mark.parametrize("kernel, pieces, T, f, d", [
    ("small", True, 129, 128, 392), ("tiles", False, 129, 128, 8), ("tiles", True, 771, 640, 1544),
    ("half", False, 1803, 1280, 392), ("half", True, 771, 1280, 1544), ("wide", False, 2049, 2176, 776),
    ("wide", True, 129, 4224, 7176)])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_int8_forms(kernel, pieces, T, f, d, name):
    """The same saved in 8 bits."""
    takes(kernel, pieces, T, 2 * f, d, "gated_int8")
    test_gpu_dense.check_ffn(T, d, f, name, "int8", name == "gelu", True)


@pytest.mark.parametrize("kernel, pieces, T, f, d", [
    ("small", False, 129, 128, 8), ("small", True, 129, 128, 3080), ("tiles", False, 3081, 2176, 136),
    ("tiles", True, 1237, 640, 7176), ("half", False, 2049, 2176, 520), ("half", True, 771, 1280, 3080),
    ("wide", False, 2049, 4224, 776), ("wide", True, 2049, 2176, 3080)])
@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("save", ["bf16", "int8"])
def test_dgated_forms(kernel, pieces, T, f, d, name, save):
    """dh with [dG, dU] and h formed on it, seen in all gradients."""
    takes(kernel, pieces, T, f, d, "gradient")
    test_gpu_dense.check_ffn(T, d, f, name, save, True, False)


@pytest.mark.parametrize("M, N, K, product", [(1, 256, 7168, "forward"), (4, 64, 64, "gated")])
def test_few_rows(M, N, K, product):
    assert ops.dense_kernel(M, N, K, product) == ("thin", 0)
    assert ops.dense_kernel(5, N, K, product)[0] == "slab" and ops.dense_kernel(128, N, K, product)[0] == "slab"


@pytest.mark.parametrize("T, K, N", [(1, 72, 30), (3, 136, 140), (4, 2056, 5000), (40, 136, 140), (128, 1032, 300),
                                     (150, 136, 140), (1500, 136, 1032), (3081, 520, 1288), (2049, 776, 2056)])
def test_nan_and_inf_stay_in_their_rows_and_columns(T, K, N):
    """Each product of a linear layer with a NaN in one row of an operand and an
    infinity in another: everything else has the bits it has without them."""
    say(f"nan T={T} K={K} N={N}")
    p = LinearPlan(T, K, N, train=True, device=DEV)
    x, W, dy = normal((T, K), 1), normal((N, K), 2, 0.1), normal((T, N), 3)

    def run():
        return [t.clone() for t in (p.forward(x, W), *p.backward(dy, x, W)[:2])]

    def others(t, dim, bad):
        keep = torch.tensor([i for i in range(t.shape[dim]) if i not in bad], dtype=torch.long, device=DEV)
        return t.index_select(dim, keep)

    clean = run()
    t0, n0, n1 = T - 1, N - 1, N // 2
    x[t0, K - 1] = float("nan")      # out: row t0; dW: column K - 1
    W[n0, 0] = float("nan")          # out: column n0; dx: column 0
    dy[0, n1] = float("inf")         # dx: row 0; dW: row n1
    out, dx, dW = run()
    assert out[t0].isnan().all() and out[:, n0].isnan().all()
    assert dx[:, 0].isnan().all() and not dx[0].isfinite().any()
    assert dW[:, K - 1].isnan().all() and not dW[n1].isfinite().any()
    for got, ref, rows, cols in ((out, clean[0], {t0}, {n0}), (dx, clean[1], {0}, {0}), (dW, clean[2], {n1}, {K - 1})):
        assert torch.equal(others(others(got, 0, rows), 1, cols), others(others(ref, 0, rows), 1, cols))
