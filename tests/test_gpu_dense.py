"""The dense products on the GPU against plain 64-bit forms, element by element
within the bounds dense_ref derives."""

import ctypes

import pytest
import torch

import dense_ref
from dense_ref import ACT_ERR, SLOPE, U16, acc_err, act, close, d64, keep8, spread
from gpu_util import DEV, say
from moe_expert_layer_r3_amd import ops
from moe_expert_layer_r3_amd.dense import GatedFFNPlan, LinearPlan

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def normal(shape, seed, std=1.0, dtype=BF, pad=0):
    """Seeded values; pad > 0: a column slice of a buffer that much wider."""
    g = torch.Generator().manual_seed(seed)
    rows, cols = shape if len(shape) == 2 else (1, shape[0])
    t = (torch.randn((rows, cols + pad), generator=g) * std).to(dtype).to(DEV)
    t = t[:, :cols] if pad else t
    return t if len(shape) == 2 else t[0]


# ---------------------------------------------------------------- linear

def check_linear(T, K, N, name, f32, bias, res, train, pad=0, std=None):
    say(f"linear T={T} K={K} N={N} act={name} f32={f32} bias={bias} res={res} pad={pad}")
    x, W = normal((T, K), 1, pad=pad), normal((N, K), 2, std or 1.7 / K ** 0.5, pad=pad)
    b = normal((N,), 3, 0.5) if bias else None
    r = normal((T, N), 4, pad=pad) if res else None
    p = LinearPlan(T, K, N, act=name, out_dtype=torch.float32 if f32 else BF, train=train, bias=bias, device=DEV)
    out = p.forward(x, W, bias=b, residual=r)
    X, Wd = d64(x), d64(W)
    z = X @ Wd.t() + (0 if b is None else d64(b))
    ez = acc_err(K, X, Wd.t()) + (0 if b is None else (K + 8) * 2.0 ** -24 * d64(b).abs())
    v, _ = act(name, z)
    ref = v + (0 if r is None else d64(r))
    e = SLOPE * ez + ACT_ERR * (z.abs() + 1) * (name != "none") + 2.0 ** -24 * ref.abs()
    close(out, ref, e + (0 if f32 else U16 * (ref.abs() + e)) + 1e-30, "out")
    if not train:
        return
    pre = z
    if p.pre is not None:
        close(p.pre, z, ez + U16 * (z.abs() + ez) + 1e-30, "pre")
        pre = d64(p.pre)
    dy = normal((T, N), 5, dtype=torch.float32 if f32 else BF)
    add = normal((T, K), 6) if res else None
    dx, dW, db = p.backward(dy, x, W, dx_add=add)
    _, slope = act(name, pre)
    dz = d64(dy) * slope
    edz = (ACT_ERR * (pre.abs() + 1) * d64(dy).abs() if name != "none" else 0 * dz)
    rdz = edz + U16 * (dz.abs() + edz) * (f32 or name != "none")   # rounded for the products
    ref = dz @ Wd + (0 if add is None else d64(add))
    e = rdz @ Wd.abs() + (N + 8) * 2.0 ** -24 * ((dz.abs() + rdz) @ Wd.abs() + (0 if add is None else d64(add).abs()))
    close(dx, ref, e + U16 * (ref.abs() + e) + 1e-30, "dx")
    ref = dz.t() @ X
    e = rdz.t() @ X.abs() + acc_err(T, dz.t().abs() + rdz.t(), X)
    close(dW, ref, e + U16 * (ref.abs() + e) + 1e-30, "dW")
    if bias:
        ref = dz.sum(0)
        e = edz.sum(0) + (T + 8) * 2.0 ** -24 * dz.abs().sum(0)
        close(db, ref, e + U16 * (ref.abs() + e) + 1e-30, "db")


@pytest.mark.parametrize("T, K, N", [(1, 8, 1), (1, 64, 256), (3, 72, 7), (16, 520, 130), (17, 256, 16), (48, 128, 512),
                                     (64, 1024, 64), (65, 200, 33), (128, 64, 128), (129, 136, 257), (203, 520, 1001),
                                     (300, 2048, 96), (513, 64, 264)])
@pytest.mark.parametrize("f32", [False, True])
def test_linear_sizes(T, K, N, f32):
    check_linear(T, K, N, "none", f32, True, False, True)


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("T, K, N, pad", [(5, 96, 40, 0), (133, 264, 77, 24), (260, 64, 300, 8)])
def test_linear_epilogue(T, K, N, pad, name):
    check_linear(T, K, N, name, False, True, True, True, pad)
    check_linear(T, K, N, name, True, False, True, True, pad)


@pytest.mark.parametrize("T, K, N", [(1, 7168, 256), (40, 7168, 256), (700, 7168, 256), (2, 2048, 7168)])
def test_linear_router_sizes(T, K, N):
    check_linear(T, K, N, "none", True, True, False, N == 256)


def test_linear_large_values():
    """Pre-activations far into the tails (|z| up to several hundred)."""
    for name in ("relu", "silu", "gelu", "sigmoid"):
        check_linear(64, 64, 64, name, True, False, False, False, std=10.0)


def test_linear_nan_and_inf_stay_in_their_rows():
    T, K, N = 150, 136, 140
    x, W = normal((T, K), 1), normal((N, K), 2)
    want = LinearPlan(T, K, N, device=DEV).forward(x, W).clone()
    x[7, 3] = float("nan")
    x[130, 135] = float("inf")
    W[139, 0] = float("nan")
    out = LinearPlan(T, K, N, device=DEV).forward(x, W)
    rows = torch.tensor([t for t in range(T) if t not in (7, 130)], device=DEV)
    assert torch.isnan(out[7]).all() and not torch.isfinite(out[130]).any() and torch.isnan(out[:, 139]).all()
    assert torch.equal(out[rows][:, :139], want[rows][:, :139])


def test_linear_writes_only_its_columns():
    """Strided output and residual in place through the C ABI: columns past N,
    rows past T and the rest of the buffer stay as they were."""
    T, K, N, ldo = 131, 72, 50, 61
    x, W = normal((T, K), 1), normal((N, K), 2)
    buf = torch.full(((T + 2) * ldo,), 7.0, dtype=BF, device=DEV)
    ref = LinearPlan(T, K, N, device=DEV).forward(x, W).clone()
    ops._call("moe_linear", ops._p(x), K, ops._p(W), K, None, ops._p(buf), ldo, T, N, K, 0, ops._p(buf), 0, ldo, None,
              None, 0, ops._stream())
    got = buf.view(T + 2, ldo)
    X, Wd = d64(x), d64(W)
    want = X @ Wd.t() + 7
    e = acc_err(K, X, Wd.t()) + (K + 8) * 2.0 ** -24 * 7
    close(got[:T, :N], want, e + U16 * (want.abs() + e), "in place")
    assert (got[:T, N:] == 7).all() and (got[T:] == 7).all() and ref.shape == (T, N)


def test_linear_empty():
    p = LinearPlan(0, 64, 24, train=True, bias=True, device=DEV)
    p.dW.fill_(3)
    p.db.fill_(3)
    x, W = torch.empty((0, 64), dtype=BF, device=DEV), normal((24, 64), 2)
    assert p.forward(x, W).shape == (0, 24)
    dx, dW, db = p.backward(torch.empty((0, 24), dtype=BF, device=DEV), x, W)
    assert dx.shape == (0, 64) and (dW == 0).all() and (db == 0).all()


@pytest.mark.parametrize("name", ["silu", "gelu", "sigmoid"])
def test_activation_slopes_against_differences(name):
    """W = identity, so out = act(z) in fp32 and dx = act'(z): central
    differences of the kernel's own values with step h = 1/16 (z on a grid of
    1/16 up to 7 is exact in bf16) differ by h^2/6 max|act'''| (< 2 for these)
    + 2 * 2^-20 * 8 / (2 h) from the values' error, and dx by two roundings."""
    h = 1 / 16
    z = torch.arange(-7, 7, h)[:216].view(27, 8)
    W = torch.eye(8).to(BF).to(DEV)
    p = LinearPlan(27, 8, 8, act=name, out_dtype=torch.float32, train=True, device=DEV)
    up = d64(p.forward((z + h).to(BF).to(DEV), W))
    dn = d64(p.forward((z - h).to(BF).to(DEV), W))
    x = z.to(BF).to(DEV)
    p.forward(x, W)
    dx, _, _ = p.backward(torch.ones(27, 8, device=DEV), x, W)
    tol = torch.full((27, 8), 2 * h * h / 6 + 2.0 ** -20 * 8 / h + 2 * U16 * SLOPE, dtype=torch.float64)
    close(dx, (up - dn) / (2 * h), tol, name)


# ---------------------------------------------------------------- gated block

def check_ffn(T, d, f, name, save, bias, res, pad=0):
    say(f"ffn T={T} d={d} f={f} act={name} save={save} bias={bias} res={res}")
    x = normal((T, d), 1, pad=pad)
    W13, W2 = normal((2 * f, d), 2, 1.7 / d ** 0.5), normal((d, f), 3, 1 / f ** 0.5)
    b13, b2 = (normal((2 * f,), 4, 0.5), normal((d,), 5, 0.5)) if bias else (None, None)
    r = normal((T, d), 6) if res else None
    p = GatedFFNPlan(T, d, f, act=name, save=save, bias=bias, device=DEV)
    y = p.forward(x, W13, W2, b13=b13, b2=b2, residual=r)
    X, A, B = d64(x), d64(W13), d64(W2)
    gu = X @ A.t() + (0 if b13 is None else d64(b13))
    e = acc_err(d, X, A.t()) + (0 if b13 is None else (d + 8) * 2.0 ** -24 * d64(b13).abs())
    G, U, eG, eU = gu[:, :f], gu[:, f:], e[:, :f], e[:, f:]
    v, _ = act(name, G)
    ev = SLOPE * eG + ACT_ERR * (G.abs() + 1)
    h = v * U
    eh = ev * U.abs() + v.abs() * eU + ev * eU
    close(p.h, h, eh + U16 * (h.abs() + eh) + 1e-30, "h")
    H = d64(p.h)
    ref = H @ B.t() + (0 if b2 is None else d64(b2)) + (0 if r is None else d64(r))
    e2 = acc_err(f, H, B.t()) + (f + 8) * 2.0 ** -24 * (ref.abs() + (0 if r is None else d64(r).abs()) + 1)
    close(y, ref, e2 + U16 * (ref.abs() + e2) + 1e-30, "y")
    if save == "none":
        return
    if save == "bf16":
        close(p.gu, gu, e + U16 * (gu.abs() + e) + 1e-30, "gu")
        kept = d64(p.gu)
    else:
        q, s = p.gu.to(X.device), p.gu_s.to(X.device)
        assert q.abs().max() <= 127
        amax = gu.abs().view(T, 2 * f // 128, 128).amax(2).t()
        worst = e.view(T, 2 * f // 128, 128).amax(2).t()
        close(s, amax / 127, worst / 127 + 2.0 ** -23 * amax / 127 + 1e-30, "gu_s")
        kept = d64(q) * d64(spread(s, 2 * f))
        # half a step, the sum's error, the factor's roundings on a value up to 127 steps
        close(kept, gu, d64(spread(s, 2 * f)) * (0.5 + 127 * 2.0 ** -21) + e + 1e-30, "gu restored")
    G, U = kept[:, :f], kept[:, f:]
    v, sl = act(name, G)
    dy, add = normal((T, d), 7), normal((T, d), 8) if res else None
    dx, dW13, dW2, db13, db2 = p.backward(dy, x, W13, W2, dx_add=add)
    DY = d64(dy)
    dh, edh = DY @ B, acc_err(d, DY, B)
    ea = ACT_ERR * (G.abs() + 1)
    dG, dU = dh * U * sl, dh * v
    eG = edh * (U * sl).abs() + (dh.abs() + edh) * U.abs() * ea
    eU = edh * v.abs() + (dh.abs() + edh) * ea
    dgu, edgu = torch.cat([dG, dU], 1), torch.cat([eG, eU], 1)
    rgu = edgu + U16 * (dgu.abs() + edgu)
    ref = dgu @ A + (0 if add is None else d64(add))
    e = rgu @ A.abs() + (2 * f + 8) * 2.0 ** -24 * ((dgu.abs() + rgu) @ A.abs() + (0 if add is None else d64(add).abs()))
    close(dx, ref, e + U16 * (ref.abs() + e) + 1e-30, "dx")
    ref = dgu.t() @ X
    e = rgu.t() @ X.abs() + acc_err(T, dgu.t().abs() + rgu.t(), X)
    close(dW13, ref, e + U16 * (ref.abs() + e) + 1e-30, "dW13")
    hh = v * U
    rh = U.abs() * ea
    rh = rh + U16 * (hh.abs() + rh)
    ref = DY.t() @ hh
    e = DY.t().abs() @ rh + acc_err(T, DY.t(), hh.abs() + rh)
    close(dW2, ref, e + U16 * (ref.abs() + e) + 1e-30, "dW2")
    if bias:
        ref = dgu.sum(0)
        e = rgu.sum(0) + (T + 8) * 2.0 ** -24 * (dgu.abs() + rgu).sum(0)
        close(db13, ref, e + U16 * (ref.abs() + e) + 1e-30, "db13")
        ref = DY.sum(0)
        e = (T + 8) * 2.0 ** -24 * DY.abs().sum(0)
        close(db2, ref, e + U16 * (ref.abs() + e) + 1e-30, "db2")


@pytest.mark.parametrize("T, d, f", [(1, 8, 8), (1, 128, 256), (2, 64, 128), (15, 264, 120), (16, 512, 64), (33, 136, 136),
                                     (64, 256, 128), (65, 72, 200), (130, 384, 392), (257, 128, 128), (300, 1032, 344)])
@pytest.mark.parametrize("save", ["none", "bf16"])
def test_ffn_sizes(T, d, f, save):
    check_ffn(T, d, f, "silu", save, False, True)


@pytest.mark.parametrize("T, d, f", [(1, 64, 128), (31, 136, 128), (64, 128, 256), (100, 64, 384), (200, 1024, 128),
                                     (3000, 64, 256)])
def test_ffn_int8(T, d, f):
    check_ffn(T, d, f, "silu", "int8", False, True)
    check_ffn(T, d, f, "gelu", "int8", True, False)


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "sigmoid"])
def test_ffn_activations(name):
    check_ffn(90, 200, 72, name, "bf16", True, True, pad=16)
    check_ffn(6, 200, 72, name, "bf16", True, False)


@pytest.mark.parametrize("T", [1, 3, 48, 200])
def test_ffn_long_sums(T):
    check_ffn(T, 4096, 2048, "silu", "none", False, True)


def test_ffn_only_h():
    """y == NULL stops after h."""
    T, d, f = 70, 64, 72
    x, W13, W2 = normal((T, d), 1), normal((2 * f, d), 2, 0.2), normal((d, f), 3)
    p = GatedFFNPlan(T, d, f, device=DEV)
    p.forward(x, W13, W2)
    h = torch.full((T + 1, f), 5.0, dtype=BF, device=DEV)
    ops._call("moe_gated_ffn", ops._p(x), d, ops._p(W13), None, None, None, None, T, d, f, 2, ops._p(h), None, 0, None,
              None, ops._p(p.ws), p.ws.numel(), ops._stream())
    assert torch.equal(h[:T], p.h) and (h[T] == 5).all()


def test_ffn_empty():
    p = GatedFFNPlan(0, 64, 128, save="int8", bias=True, device=DEV)
    for t in (p.dW13, p.dW2, p.db13, p.db2):
        t.fill_(3)
    x, W13, W2 = torch.empty((0, 64), dtype=BF, device=DEV), normal((256, 64), 2), normal((64, 128), 3)
    p.forward(x, W13, W2)
    p.backward(x, x, W13, W2)
    assert all((t == 0).all() for t in (p.dW13, p.dW2, p.db13, p.db2))


def test_ffn_gradient_against_differences():
    """Directional differences of the 64-bit loss sum(dy * y) along random
    directions of x, W13 and W2 (step 1e-4, so their own error is far below the
    bound) against the kernels' gradients: |<got - exact, v>| <= sum tol |v| with
    the roundings of dgu / h (2^-8 of each summand) and of the result."""
    T, d, f = 12, 40, 24
    x, W13, W2, dy = normal((T, d), 1), normal((2 * f, d), 2, 0.3), normal((d, f), 3, 0.2), normal((T, d), 4)
    p = GatedFFNPlan(T, d, f, save="bf16", device=DEV)
    p.forward(x, W13, W2)
    grads = p.backward(dy, x, W13, W2)[:3]
    val = [d64(x), d64(W13), d64(W2)]
    DY = d64(dy)

    def loss(X, A, B):
        gu = X @ A.t()
        v, _ = act("silu", gu[:, :f])
        return (DY * ((v * gu[:, f:]) @ B.t())).sum()

    # the saved gu is rounded too: slopes and factors move by 2^-8 relative to |G|, |U|
    gen = torch.Generator().manual_seed(9)
    for i, got in enumerate(grads):
        for _ in range(4):
            v = torch.randn(val[i].shape, generator=gen, dtype=torch.float64)
            eps = 1e-4
            up = [t + (eps * v if j == i else 0) for j, t in enumerate(val)]
            dn = [t - (eps * v if j == i else 0) for j, t in enumerate(val)]
            want = (loss(*up) - loss(*dn)) / (2 * eps)
            G = d64(got)
            # three roundings in a row (gu, dgu or h, the result), each at most 2^-8 of summands
            # whose magnitudes add up to the same products of absolute values
            X, A, B = (t.abs() for t in val)
            gu = X @ A.t()
            mag_dh = DY.abs() @ B
            mag = torch.cat([mag_dh * gu[:, f:] * (SLOPE + gu[:, :f]), mag_dh * gu[:, :f] * SLOPE], 1)
            m = [mag @ A, mag.t() @ X, DY.abs().t() @ (gu[:, :f] * gu[:, f:] * SLOPE)][i]
            tol = 3 * U16 * 1.01 * (m * v.abs()).sum()
            assert abs((G * v).sum() - want) <= tol, (i, float((G * v).sum()), float(want), float(tol))


# ---------------------------------------------------------------- 256 x 256 tiles

@pytest.fixture
def on_gpu():
    dense_ref.REF[0] = DEV
    yield
    dense_ref.REF[0] = "cpu"


@pytest.mark.parametrize("T, K, N", [(3300, 200, 4200), (3300, 4200, 72), (100, 4200, 3304), (64, 4104, 3301),
                                     (4096, 64, 4096), (2305, 8, 5000), (3841, 136, 3841)])
def test_linear_wide(on_gpu, T, K, N):
    """Forward, data- and weight-gradient products of at least 192 tiles in turn;
    K from less than one step to several, odd and even numbers of steps."""
    check_linear(T, K, N, "silu", False, True, True, True, pad=8)
    check_linear(T, K, N, "none", True, False, False, True)


@pytest.mark.parametrize("T, K, N", [(8192, 7168, 256), (1500, 7168, 3000)])
def test_linear_wide_pieces(on_gpu, T, K, N):
    """256 x 256 tiles with K in pieces, forward and weight gradient."""
    check_linear(T, K, N, "none", True, True, False, True)


@pytest.mark.parametrize("save", ["bf16", "int8"])
def test_ffn_wide_pieces(on_gpu, save):
    check_ffn(1100, 7168, 2048, "silu", save, True, True)


@pytest.mark.parametrize("T, d, f, save", [(3300, 72, 2104, "bf16"), (3300, 200, 4200, "bf16"), (3300, 136, 2176, "int8"),
                                           (3300, 64, 4224, "int8"), (6000, 1000, 1032, "none")])
def test_ffn_wide(on_gpu, T, d, f, save):
    check_ffn(T, d, f, "silu", save, save == "bf16", True)
    check_ffn(T, d, f, "gelu", save, False, False)


# ---------------------------------------------------------------- what must stay untouched, offsets past 32 bits

class Guarded:
    """Output buffers with 4096 poisoned elements in front and behind."""

    def __init__(self):
        self.bufs = []

    def __call__(self, shape, dtype=BF):
        n = 1
        for v in shape:
            n *= v
        n16 = (n + 7) // 8 * 8
        b = torch.full((n16 + 8192,), 77, dtype=dtype, device=DEV)
        self.bufs.append((b, n))
        return b[4096:4096 + n]

    def check(self):
        for b, n in self.bufs:
            assert (b[:4096] == 77).all() and (b[4096 + n:] == 77).all()


@pytest.mark.parametrize("T, d, f", [(3, 72, 136), (37, 136, 128), (131, 200, 136), (700, 1032, 520), (3300, 72, 2184),
                                     (3300, 2056, 4104)])
@pytest.mark.parametrize("save", ["bf16", "int8"])
def test_nothing_past_the_outputs(T, d, f, save):
    if save == "int8":
        f = f // 128 * 128
    g = Guarded()
    p = lambda t: t.data_ptr()
    x, W13, W2, dy = normal((T, d), 1), normal((2 * f, d), 2, 0.1), normal((d, f), 3, 0.1), normal((T, d), 4)
    h, y, dx, dW13, dW2, db13, db2 = g((T, f)), g((T, d)), g((T, d)), g((2 * f, d)), g((d, f)), g((2 * f,)), g((d,))
    gu = g((T, 2 * f), BF if save == "bf16" else torch.int8)
    gs = g((2 * f // 128, T), torch.float32) if save == "int8" else None
    nb = max(ops.workspace_bytes("moe_gated_ffn_workspace", T, d, f),
             ops.workspace_bytes("moe_gated_ffn_backward_workspace", T, d, f))
    ws = g((nb,), torch.uint8)
    gp = None if gs is None else p(gs)
    ops.launch("moe_gated_ffn", x.device, p(x), d, p(W13), None, p(W2), None, p(dy), T, d, f, 2, p(h), p(y),
               ops.SAVES[save], p(gu), gp, p(ws), nb)
    ops.launch("moe_gated_ffn_backward", x.device, p(dy), p(x), d, p(W13), p(W2), ops.SAVES[save], p(gu), gp, None, T, d, f,
               2, p(dx), p(dW13), p(dW2), p(db13), p(db2), p(ws), nb)
    # a linear layer with an odd number of columns on the same inputs
    N = 2 * f - 3
    out, pre, lx, lW, lb = g((T, N)), g((T, N)), g((T, d)), g((N, d)), g((N,))
    nl = max(ops.workspace_bytes("moe_linear_workspace", T, N, d), ops.workspace_bytes("moe_linear_backward_workspace", T, N, d))
    wl = g((nl,), torch.uint8)
    ops.launch("moe_linear", x.device, p(x), d, p(W13), d, None, None, N, T, N, d, 3, p(out), 0, N, p(pre), p(wl), nl)
    ops.launch("moe_linear_backward", x.device, p(out), 0, p(pre), p(x), d, p(W13), d, None, T, N, d, 3, p(lx), p(lW), p(lb),
               p(wl), nl)
    torch.cuda.synchronize()
    g.check()


def test_offsets_past_32_bits():
    """x of 2.2e9 elements and an output of 2.2e9: rows at the far end against
    the same rows alone, and the weight gradient against the sum of two halves."""
    T, K, N = 307_203, 7168, 8
    x = torch.randn((T, K), device=DEV, dtype=BF)
    W, dy = normal((N, K), 2, 0.02), normal((T, N), 3)
    p = LinearPlan(T, K, N, train=True, device=DEV)
    out = p.forward(x, W)
    X, Wd = x[-200:].double(), W.double()
    ref = X @ Wd.t()
    e = acc_err(K, X, Wd.t())
    assert ((out[-200:].double() - ref).abs() <= e + U16 * (ref.abs() + e)).all()
    dx, dW, _ = p.backward(dy, x, W)
    D = dy[-200:].double()
    ref = D @ Wd
    e = acc_err(N, D, Wd)
    assert ((dx[-200:].double() - ref).abs() <= e + U16 * (ref.abs() + e) + 1e-30).all()
    ref = sum(dy[a:a + 50_000].double().t() @ x[a:a + 50_000].double() for a in range(0, T, 50_000))
    mag = sum(dy[a:a + 50_000].double().abs().t() @ x[a:a + 50_000].double().abs() for a in range(0, T, 50_000))
    e = (T + 8) * 2.0 ** -24 * mag
    assert ((dW.double() - ref).abs() <= e + U16 * (ref.abs() + e)).all()
    del p, out, dx
    q, s = ops.act_save(x)
    back = ops.act_restore(q, s)
    q1, s1 = ops.act_save(x[-200:])
    assert torch.equal(q[-200:], q1) and torch.equal(s[:, -200:], s1)
    assert torch.equal(back[-200:], ops.act_restore(q1, s1))
    del x, q, s, back
    x, W = normal((T, 16), 4), normal((K, 16), 5)   # an output of 2.2e9 elements
    out = LinearPlan(T, 16, K, device=DEV).forward(x, W)
    X, Wd = x[-200:].double(), W.double()
    ref = X @ Wd.t()
    e = acc_err(16, X, Wd.t())
    assert ((out[-200:].double() - ref).abs() <= e + U16 * (ref.abs() + e) + 1e-30).all()


def ints(shape, seed):
    """-1, 0 and 1: every sum of the tests that use them is exact in fp32, whatever its order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-1, 2, shape, device=DEV, generator=g).to(BF)


@pytest.mark.parametrize("T, d, f", [(2, 72, 40), (90, 72, 136), (700, 72, 136), (1237, 520, 264), (3300, 520, 264)])
def test_gradients_one_by_one(T, d, f):
    """Each gradient alone and without the others, against all at once."""
    p = lambda t: None if t is None else t.data_ptr()
    x, W13, W2, dy, W = ints((T, d), 1), ints((2 * f, d), 2), ints((d, f), 3), ints((T, d), 4), ints((f, d), 5)
    plan = GatedFFNPlan(T, d, f, act="relu", save="bf16", bias=True, device=DEV)
    plan.forward(x, W13, W2)
    want = [t.clone() for t in plan.backward(dy, x, W13, W2)]
    assert torch.equal(want[4], dy.double().sum(0).to(BF))
    n = len(want)
    for on in [{i} for i in range(n)] + [set(range(n)) - {i} for i in range(n)] + [{1, 2}, {3, 4}, {0, 4}]:
        out = [torch.empty_like(t) if i in on else None for i, t in enumerate(want)]
        ops.launch("moe_gated_ffn_backward", x.device, p(dy), p(x), d, p(W13), p(W2), 1, p(plan.gu), None, None, T, d, f, 1,
                   *map(p, out), p(plan.ws), plan.ws_bytes)
        assert all(t is None or torch.equal(t, w) for t, w in zip(out, want)), on
    dz = ints((T, f), 6)
    plan = LinearPlan(T, d, f, train=True, bias=True, device=DEV)
    want = [t.clone() for t in plan.backward(dz, x, W)]
    for a, b in zip(want, (dz.double() @ W.double(), dz.double().t() @ x.double(), dz.double().sum(0))):
        assert torch.equal(a, b.to(BF))
    for on in ({0}, {1}, {2}, {0, 1}, {0, 2}, {1, 2}):
        out = [torch.empty_like(t) if i in on else None for i, t in enumerate(want)]
        ops.launch("moe_linear_backward", x.device, p(dz), 0, None, p(x), d, p(W), d, None, T, f, d, 0, *map(p, out),
                   p(plan.ws), plan.ws_bytes)
        assert all(t is None or torch.equal(t, w) for t, w in zip(out, want)), on


def test_most_rows():
    """2^30 rows, the most there may be: blocks of rows repeat, and so do the results."""
    T, R = 1 << 30, 1 << 20
    b = normal((R, 8), 1)
    x, W = b.repeat(T // R, 1), normal((8, 8), 2)
    same = lambda t, ref: all(torch.equal(v, ref) for v in t.view(T // R, R, *t.shape[1:]))
    p = LinearPlan(T, 8, 8, device=DEV)
    out = p.forward(x, W)
    assert torch.equal(out[:R], LinearPlan(R, 8, 8, device=DEV).forward(b, W)) and same(out, out[:R])
    del p, out
    p = GatedFFNPlan(T, 8, 8, device=DEV)
    W13, W2 = normal((16, 8), 3), normal((8, 8), 4)
    y = p.forward(x, W13, W2)
    assert torch.equal(y[:R], GatedFFNPlan(R, 8, 8, device=DEV).forward(b, W13, W2)) and same(y, y[:R])
    del p, y
    q, s = ops.act_save(x)
    q1, s1 = ops.act_save(b)
    assert same(q, q1) and same(s[0], s1[0])
    assert same(ops.act_restore(q, s), ops.act_restore(q1, s1))


@pytest.mark.parametrize("T", [1, 3, 100, 700, 3300])
def test_in_place(T):
    """The addend's memory as the output's."""
    d, f = 520, 264
    x, W13, W2, W = normal((T, d), 1), normal((2 * f, d), 2, 0.1), normal((d, f), 3, 0.1), normal((d, d), 4, 0.1)
    r, dy = normal((T, d), 5), normal((T, d), 6)
    p, q = LinearPlan(T, d, d, train=True, device=DEV), GatedFFNPlan(T, d, f, save="bf16", device=DEV)
    for plan, out, fwd, bwd in ((p, p.out, (x, W), (dy, x, W)), (q, q.y, (x, W13, W2), (dy, x, W13, W2))):
        want = plan.forward(*fwd, residual=r).clone()
        out.copy_(r)
        assert torch.equal(plan.forward(*fwd, residual=out), want)
        want = plan.backward(*bwd, dx_add=r)[0].clone()
        plan.dx.copy_(r)
        assert torch.equal(plan.backward(*bwd, dx_add=plan.dx)[0], want)


# ---------------------------------------------------------------- 8-bit activations

@pytest.mark.parametrize("rows, cols, pad", [(1, 8, 0), (3, 128, 0), (5, 136, 24), (130, 1000, 0), (257, 384, 8),
                                             (1024, 7168, 0)])
def test_act8_bits(rows, cols, pad):
    g = torch.Generator().manual_seed(rows)
    x = torch.randn((rows, cols + pad), generator=g) * torch.exp(3 * torch.randn((rows, 1), generator=g))
    x[0, 0] = 1e-40   # a subnormal bf16
    if rows > 2:
        x[1] = 0      # an empty block
        x[2, ::2] *= 1e30
    x = x.to(BF).to(DEV)[:, :cols]
    q, s = ops.act_save(x)
    wq, ws = keep8(x.cpu().float())
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.cpu().float(), wq)
    back = ops.act_restore(q, s)
    assert torch.equal(back.cpu(), (wq * spread(ws, cols)).to(BF))


def test_act8_nan_and_inf():
    x = normal((6, 256), 3)
    clean = ops.act_restore(*ops.act_save(x))
    x[1, 5], x[3, 200], x[5, 0] = float("nan"), float("inf"), float("-inf")
    back = ops.act_restore(*ops.act_save(x))
    bad = torch.zeros(6, 256, dtype=torch.bool, device=DEV)
    bad[1, :128] = bad[3, 128:] = bad[5, :128] = True
    assert torch.isnan(back[bad]).all() and torch.equal(back[~bad], clean[~bad])


def test_act8_empty():
    x = torch.empty((0, 128), dtype=BF, device=DEV)
    q, s = ops.act_save(x)
    assert ops.act_restore(q, s).shape == (0, 128)


# ---------------------------------------------------------------- streams, graphs, repeated runs

def test_same_bits_every_time_and_on_another_stream():
    T, d, f = 333, 512, 256
    x, W13, W2, dy = normal((T, d), 1), normal((2 * f, d), 2, 0.1), normal((d, f), 3, 0.1), normal((T, d), 4)
    p = GatedFFNPlan(T, d, f, save="int8", bias=True, device=DEV)

    def once():
        y = p.forward(x, W13, W2, residual=dy)
        return [t.clone() for t in (y, *p.backward(dy, x, W13, W2))]

    a = once()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = once()
    torch.cuda.synchronize()
    for s, t in zip(a, b):
        assert torch.equal(s, t)


def test_graph_replays():
    """Forward and backward of both plans in one graph, replayed between eager
    passes on the same buffers with other inputs."""
    from moe_expert_layer_r3_amd.layer import capture_graph
    T, d, f, E = 200, 256, 128, 64
    x, W13, W2, dy = normal((T, d), 1), normal((2 * f, d), 2, 0.1), normal((d, f), 3, 0.1), normal((T, d), 4)
    Wr, dl = normal((E, d), 5, 0.1), normal((T, E), 6, dtype=torch.float32)
    p = GatedFFNPlan(T, d, f, save="int8", device=DEV)
    r = LinearPlan(T, d, E, out_dtype=torch.float32, train=True, device=DEV)

    def step():
        lg = r.forward(x, Wr)
        y = p.forward(x, W13, W2, residual=dy)
        g = r.backward(dl, x, Wr)
        return [lg, y, *g[:2], *p.backward(dy, x, W13, W2, dx_add=g[0])[:3]]

    graph = capture_graph(step)
    for i in range(4):
        x.copy_(normal((T, d), 20 + i))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in (r.out, p.y, r.dx, r.dW, p.dx, p.dW13, p.dW2):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (r.out, p.y, r.dx, r.dW, p.dx, p.dW13, p.dW2)):
            assert torch.equal(a, b)


def test_two_plans_at_once():
    """Two plans (own workspaces) on two streams give what each gives alone."""
    T, K, N = 40, 4096, 64
    xs = [normal((T, K), i) for i in range(2)]
    W = normal((N, K), 9, 0.05)
    ps = [LinearPlan(T, K, N, out_dtype=torch.float32, device=DEV) for _ in range(2)]
    want = [p.forward(x, W).clone() for p, x in zip(ps, xs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, p, x in zip(streams, ps, xs):
            with torch.cuda.stream(s):
                p.forward(x, W)
    torch.cuda.synchronize()
    for p, w in zip(ps, want):
        assert torch.equal(p.out, w)


def test_plan_refusals():
    x, W = normal((4, 64), 1), normal((8, 64), 2)
    p = LinearPlan(4, 64, 8, device=DEV)
    with pytest.raises(ValueError):
        p.forward(x[:3], W)
    with pytest.raises(TypeError):
        p.forward(x.float(), W)
    with pytest.raises(ValueError):
        p.forward(x, W, bias=torch.zeros(8, dtype=BF))  # on the host
    with pytest.raises(ops.MoeError):
        p.forward(normal((4, 68), 1)[:, :64], W)        # rows 136 bytes apart
    with pytest.raises(ValueError):
        p.backward(p.out, x, W)                         # not a training plan
    with pytest.raises(ValueError):
        LinearPlan(4, 64, 8, act="swish", device=DEV)
    with pytest.raises(ValueError):
        GatedFFNPlan(4, 64, 72, save="int8", device=DEV)
    with pytest.raises(ops.MoeError):
        GatedFFNPlan(4, 60, 72, device=DEV)
