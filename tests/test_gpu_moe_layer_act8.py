"""What MoELayerPlan(act8=True) holds, and its steps beside one another."""

import pytest
import torch

from gpu_util import DEV
from moe_expert_layer_r3_amd import ops
from moe_expert_layer_r3_amd.dense import MoELayerPlan
from moe_expert_layer_r3_amd.layer import quantize_weights
from test_gpu_moe_layer import inputs, normal

pytestmark = pytest.mark.gpu


def held(act8, T, d, f, E, k, fs):
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    p = MoELayerPlan(T, d, f, E, k, fs, act8=act8, device=DEV)
    n = torch.cuda.memory_allocated() - before
    del p
    return n


@pytest.mark.parametrize("k", [1, 2])
def test_memory_held(k):
    """x costs one byte and 1/32 a value, [G, U] one byte and 1/32 instead of two;
    nothing else differs (allocations are rounded up to 512 bytes)."""
    T, d, f, E, fs = 4096, 512, 256, 8, 128
    more = held(True, T, d, f, E, k, fs) - held(False, T, d, f, E, k, fs)
    want = T * d * 33 // 32 + T * 2 * fs * 33 // 32 - T * 2 * fs * 2
    assert abs(more - want) <= 8 * 512, (more, want)


def test_two_backwards_and_two_layers():
    """A backward repeated, and two plans' steps in turn, give the same bits as one
    plan's alone; x itself may be gone by then."""
    T, d, f, E, k, fs = 200, 256, 128, 16, 1, 256
    a, b = inputs(T, d, f, E, fs), inputs(T, d, f, E, fs)
    b["x"], b["dy"] = normal((T, d), 21), normal((T, d), 22)
    ps = [MoELayerPlan(T, d, f, E, k, fs, act8=True, device=DEV) for _ in range(2)]
    wts = quantize_weights(a["W13"], a["W2"], transpose=ps[0].routed.transpose_weights)
    fwd = lambda p, i: p.forward(i["x"], i["Wr"], wts, i["W13s"], i["W2s"]).clone()
    bwd = lambda p, i: {n: t.clone() for n, t in p.backward(i["dy"], None, i["Wr"], wts, i["W13s"], i["W2s"]).items()
                        if t is not None}
    want = []
    for i in (a, b):
        want.append((fwd(ps[0], i), bwd(ps[0], i)))
    ys = [fwd(p, i) for p, i in zip(ps, (a, b))]
    x8 = ops.act_restore(*ops.act_save(a["x"]))
    a["x"].zero_()
    for p, i, (y, g), got in zip(ps, (a, b), want, ys):
        assert torch.equal(got, y)
        for _ in range(2):
            h = bwd(p, i)
            assert h.keys() == g.keys() and all(torch.equal(h[n], g[n]) for n in g)
    assert torch.equal(ps[0].xr, x8)
