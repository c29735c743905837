"""The dense products' kernels that only large or particular sizes take, against
plain 64-bit forms, within the bounds dense_ref derives."""

import pytest
import torch

import dense_ref
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
