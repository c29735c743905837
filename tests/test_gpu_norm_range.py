"""Norms of rows next to the end of fp32's range: a row has its norm as long as its mean
square is a number there, and rho = 0 beyond.  Bounds as norm_ref derives them."""

import pytest
import torch

import norm_ref as R
from gpu_util import DEV, say
from moe_expert_layer_r3_amd.block import JoinPlan, NormPlan
from test_gpu_norm import BF, EPS, F32, T_OF, check_norm, normal

pytestmark = pytest.mark.gpu
# root mean squares: the last three have squares, sums of squares and their mean past the range in turn
SIZES = (1.0, 1e15, 2.5e17, 4e18, 1.5e19)
OVER = 2.5e19


def rows(d, dtype, sizes):
    x = normal((len(sizes), d), 31, 1.0, F32)
    x = x / x.double().square().mean(dim=1, keepdim=True).sqrt().float()
    return (x * torch.tensor(sizes, device=DEV)[:, None]).to(dtype)


@pytest.mark.parametrize("d", [8, 64, 512, 1032, 7168, 8192, 12296, 16384, 16400, 1 << 17])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_norm_of_large_rows(d, kind):
    check_norm(len(SIZES), d, kind, "f32", x=rows(d, T_OF[kind], SIZES), add=True)


@pytest.mark.parametrize("d", [8, 1032, 7168, 12296, 16400])
def test_norm_beyond_the_range(d):
    x = rows(d, F32, (OVER, 1.0))
    p = NormPlan(2, d, x_dtype=F32, train=True, device=DEV)
    w = normal((d,), 2, 0.3, BF, 1.0)
    h = p.forward(x, w)
    dx, _ = p.backward(normal((2, d), 3), x, w)
    assert not bool(h[0].any()) and not bool(dx[0].any()) and bool(h[1].any()) and bool(dx[1].any())


@pytest.mark.parametrize("d", [64, 1032, 7168, 12296, 16400])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_join_of_large_rows(d, kind):
    """The norm behind the layer and the one in front of the next, of rows in turn."""
    say(f"join of large rows d={d} r={kind}")
    y, r = rows(d, BF, SIZES), rows(d, T_OF[kind], SIZES[::-1])
    wp, wn = normal((d,), 13, 0.3, F32, 1.0), normal((d,), 14, 0.3, F32, 1.0)
    p = JoinPlan(len(SIZES), d, r_dtype=T_OF[kind], w_dtype=F32, eps=EPS, device=DEV)
    r_out, h = p.forward(y, r, w_post=wp, w_pre=wn)
    n, _ = R.norm(R.d64(y), R.d64(wp), EPS)
    want, e = R.d64(r) + n, n.abs() * (R.rho_err(d) + R.CHAIN * R.U)
    R.close(r_out, want, e + 2 * R.U * (want.abs() + R.d64(r).abs()), "r_out")
    ref, _ = R.norm(R.d64(r_out), R.d64(wn), EPS)
    R.close(h, ref, ref.abs() * (R.rho_err(d) + R.CHAIN * R.U), "h")
