"""A layer's training step: router, routed experts and shared expert together
(MoELayerPlan), each link checked on the values the links before it produced:
the dense ones against 64-bit forms, the routed ones bit for bit against a
TrainPlan of their own."""

import pytest
import torch

from dense_ref import U16, acc_err, act, close, d64, spread
from gpu_util import DEV, say
from moe_expert_layer_r3_amd import ops
from moe_expert_layer_r3_amd.dense import MoELayerPlan
from moe_expert_layer_r3_amd.layer import TrainPlan, capture_graph, quantize_weights

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def normal(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def inputs(T, d, f, E, fs):
    return dict(x=normal((T, d), 1), dy=normal((T, d), 2), Wr=normal((E, d), 3, 2 / d ** 0.5), br=normal((E,), 4, 0.1),
                W13=normal((E, 2 * f, d), 5, 1 / d ** 0.5), W2=normal((E, d, f), 6, 1 / f ** 0.5),
                W13s=normal((2 * fs, d), 7, 1 / d ** 0.5), W2s=normal((d, fs), 8, 1 / fs ** 0.5))


@pytest.mark.parametrize("T, d, f, E, k, fs, act8", [(128, 128, 256, 8, 2, 128, False), (200, 256, 128, 16, 4, 256, True),
                                                     (1, 128, 128, 8, 2, 128, True), (77, 256, 256, 8, 8, 136, False)])
def test_layer_step(T, d, f, E, k, fs, act8):
    say(f"layer T={T} d={d} f={f} E={E} k={k} fs={fs} act8={act8}")
    a = inputs(T, d, f, E, fs)
    p = MoELayerPlan(T, d, f, E, k, fs, act8=act8, router_bias=True, device=DEV)
    wts = quantize_weights(a["W13"], a["W2"], transpose=p.routed.transpose_weights)
    y = p.forward(a["x"], a["Wr"], wts, a["W13s"], a["W2s"], br=a["br"])
    g = p.backward(a["dy"], None if act8 else a["x"], a["Wr"], wts, a["W13s"], a["W2s"])

    X, Wr = d64(a["x"]), d64(a["Wr"])
    lg = X @ Wr.t() + d64(a["br"])
    close(p.router.out, lg, acc_err(d, X, Wr.t()) + (d + 8) * 2.0 ** -24 * (lg.abs() + 1), "logits")
    # the routed experts on these logits, alone
    q = TrainPlan(T, d, f, E, E, k, device=DEV)
    yr = q.forward(a["x"], p.router.out, wts)
    dxr, dW13, dW2, dl = q.backward(a["x"], a["dy"], wts)
    for got, want in ((p.routed.y, yr), (p.routed.dx, dxr), (g["dW13"], dW13), (g["dW2"], dW2), (p.routed.d_logits, dl)):
        assert torch.equal(got, want)
    # shared expert on top
    H, B = d64(p.shared.h), d64(a["W2s"])
    ref = H @ B.t() + d64(yr)
    e = acc_err(fs, H, B.t()) + (fs + 8) * 2.0 ** -24 * d64(yr).abs()
    close(y, ref, e + U16 * (ref.abs() + e), "y")
    # router gradients with the routed experts' dx added
    xb = a["x"] if not act8 else p.xr
    if act8:
        assert torch.equal(xb, ops.act_restore(*ops.act_save(a["x"])))
    Xb, DL = d64(xb), d64(dl)
    r = U16 * DL.abs()   # dz is rounded for the products
    ref = DL @ Wr + d64(dxr)
    e = r @ Wr.abs() + (E + 8) * 2.0 ** -24 * ((DL.abs() + r) @ Wr.abs() + d64(dxr).abs())
    close(p.router.dx, ref, e + U16 * (ref.abs() + e) + 1e-30, "dx after the router")
    ref = DL.t() @ Xb
    e = r.t() @ Xb.abs() + acc_err(T, DL.t().abs() + r.t(), Xb)
    close(g["dWr"], ref, e + U16 * (ref.abs() + e) + 1e-30, "dWr")
    # the shared expert's data gradient with those added
    gu = d64(p.shared.gu) * (d64(spread(p.shared.gu_s.cpu(), 2 * fs)) if act8 else 1)
    G, U = gu[:, :fs], gu[:, fs:]
    v, sl = act("silu", G)
    dh = d64(a["dy"]) @ B
    dgu = torch.cat([dh * U * sl, dh * v], 1)
    mag = torch.cat([(d64(a["dy"]).abs() @ B.abs()) * U.abs() * 1.1, (d64(a["dy"]).abs() @ B.abs()) * v.abs()], 1)
    rd = U16 * dgu.abs() * 1.01 + 2.0 ** -18 * mag
    A = d64(a["W13s"])
    ref = dgu @ A + d64(p.router.dx)
    e = rd @ A.abs() + (2 * fs + 8) * 2.0 ** -24 * ((dgu.abs() + rd) @ A.abs() + d64(p.router.dx).abs())
    close(g["dx"], ref, e + U16 * (ref.abs() + e) + 1e-30, "dx")


@pytest.mark.parametrize("act8", [False, True])
def test_layer_graph(act8):
    """The whole step as a HIP graph, replayed on new inputs between eager runs."""
    T, d, f, E, k, fs = 160, 256, 256, 8, 2, 256
    a = inputs(T, d, f, E, fs)
    p = MoELayerPlan(T, d, f, E, k, fs, act8=act8, device=DEV)
    wts = quantize_weights(a["W13"], a["W2"], transpose=p.routed.transpose_weights)

    def step():
        y = p.forward(a["x"], a["Wr"], wts, a["W13s"], a["W2s"])
        g = p.backward(a["dy"], a["x"], a["Wr"], wts, a["W13s"], a["W2s"])
        return [y] + [t for t in g.values() if t is not None]

    graph = capture_graph(step)
    outs = step()
    for i in range(4):
        a["x"].copy_(normal((T, d), 30 + i))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for s, t in zip(want, outs):
            assert torch.equal(s, t)
