"""Blocks of a model as they are used: norm, router, scored choice, routed and
shared experts, join, twice in a row with gradients back through both; each link
checked on the values that the links around it produced (the experts' products
have tests of their own)."""

import numpy as np
import pytest
import torch

import norm_ref as N
import scores_ref as R
from gpu_util import DEV, np64, npi, say
from moe_expert_layer_r3_amd import ops
from moe_expert_layer_r3_amd.block import MoEBlockPlan, NormPlan
from moe_expert_layer_r3_amd.dense import MoELayerPlan
from moe_expert_layer_r3_amd.layer import ForwardPlan, TrainPlan, capture_graph, quantize_weights
from test_gpu_moe_layer import inputs, normal
from test_gpu_scores import close

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U16 = 2.0 ** -8


def check_route(plan, logits, sc, bias, record=None):
    """The routed plan's ids, weights and d_logits against 64-bit forms of its own logits and gate gradients."""
    l = np64(logits)
    s = R.scores(l, "f32", sc.score)
    ids = R.choice(l, s, "f32", plan.k, None if bias is None else npi(bias), sc.groups, sc.top_groups, sc.group_top) \
        if record is None else record
    assert np.array_equal(npi(plan.ids), ids)
    E = l.shape[1]
    w, _ = R.weights(l, s, "f32", ids, sc.score, sc.renorm, sc.scale)
    close(plan.w, w, (R.ROUND["f32"] + R.row_err(E, sc.score, sc.renorm)) * np.abs(w) + R.TINY["f32"], "w")
    return l, s, ids


def check_route_back(plan, l, s, ids, sc):
    g, size = R.gradient(l, s, "f32", ids, np64(plan.d_gate), sc.score, sc.renorm, sc.scale)
    close(plan.d_logits, g, R.ROUND["f32"] * np.abs(g) + R.TINY["f32"] + 2.0 ** -46 * size, "d_logits")


@pytest.mark.parametrize("T,d,f,E,k,fs,act8,r_dtype,gate", [
    (96, 256, 256, 16, 4, 256, False, BF, "channel"), (130, 128, 128, 64, 8, 128, True, F32, "token"),
    (1, 128, 256, 16, 2, 128, False, F32, "none")])
def test_two_blocks(T, d, f, E, k, fs, act8, r_dtype, gate):
    say(f"blocks T={T} d={d} f={f} E={E} k={k} fs={fs} act8={act8} {r_dtype} gate={gate}")
    sc = ops.Scoring("sigmoid", groups=4, top_groups=2, scale=2.5)
    a = [inputs(T, d, f, E, fs) for _ in range(2)]
    r0 = normal((T, d), 50, 1.0, r_dtype)
    shape = dict(none=None, channel=(d,), token=(T,))[gate]
    w = {n: (torch.randn(d, generator=torch.Generator().manual_seed(i)) * 0.2 + 1).to(BF).to(DEV)
         for i, n in enumerate(("in", "post0", "next0", "post1"))}
    gates = [None if shape is None else (torch.randn(shape, generator=torch.Generator().manual_seed(70 + i))).to(F32).to(DEV)
             for i in range(2)]
    bias = (torch.randn(E, generator=torch.Generator().manual_seed(80)) * 0.05).to(DEV)
    load = torch.zeros(E, dtype=torch.int32, device=DEV)
    kw = dict(scoring=sc, act8=act8, r_dtype=r_dtype, post=True, gate=gate, gate_dtype=F32,
              gate_act="none" if gate == "none" else "sigmoid", r_scale=0.9, y_scale=0.5)
    first = NormPlan(T, d, x_dtype=r_dtype, train=True, device=DEV)
    b = [MoEBlockPlan(T, d, f, E, k, fs, next_norm=i == 0, device=DEV, **kw) for i in range(2)]
    wts = [quantize_weights(x["W13"], x["W2"], transpose=b[0].layer.routed.transpose_weights) for x in a]
    for p in b:
        p.layer.routed.route_bias, p.layer.routed.load = bias, load
    h0 = first.forward(r0, w["in"])
    r1, h1 = b[0].forward(r0, h0, a[0]["Wr"], wts[0], a[0]["W13s"], a[0]["W2s"], w_post=w["post0"], gate=gates[0],
                          w_next=w["next0"])
    r2, h2 = b[1].forward(r1, h1, a[1]["Wr"], wts[1], a[1]["W13s"], a[1]["W2s"], w_post=w["post1"], gate=gates[1])
    assert h2 is None and int(load.sum()) == 2 * T * k
    d2 = normal((T, d), 51, 1.0, r_dtype)
    g1 = b[1].backward(d2, None, None if act8 else h1, a[1]["Wr"], wts[1], a[1]["W13s"], a[1]["W2s"], w_post=w["post1"],
                       gate=gates[1])
    g0 = b[0].backward(g1["dr"], g1["dh"], None if act8 else h0, a[0]["Wr"], wts[0], a[0]["W13s"], a[0]["W2s"],
                       w_post=w["post0"], gate=gates[0], w_next=w["next0"])
    dr, dw_in = first.backward(g0["dh"], r0, w["in"], dx_add=g0["dr"])

    # the layer between is a MoELayerPlan of its own, bit for bit
    alone = MoELayerPlan(T, d, f, E, k, fs, act8=act8, scoring=sc, device=DEV)
    alone.routed.route_bias = bias
    y = alone.forward(h0, a[0]["Wr"], wts[0], a[0]["W13s"], a[0]["W2s"])
    assert torch.equal(y, b[0].layer.shared.y)
    want = alone.backward(b[0].join.dy, None if act8 else h0, a[0]["Wr"], wts[0], a[0]["W13s"], a[0]["W2s"])
    for n, t in want.items():
        if t is not None:
            assert torch.equal(t, g0["dh" if n == "dx" else n]), n

    rounded = 2.0 ** -24 if r_dtype == F32 else U16
    for i, (p, g, rin, rout) in enumerate(((b[0], g0, r0, r1), (b[1], g1, r1, r2))):
        l, s, ids = check_route(p.layer.routed, p.layer.router.out, sc, bias)
        check_route_back(p.layer.routed, l, s, ids, sc)
        # the join: r_out from y and r
        Y, X = N.d64(p.layer.shared.y), N.d64(rin)
        n, rho = N.norm(Y, N.d64(w[f"post{i}"]), 1e-6)
        v, _ = N.gate_of(gates[i], gate, kw["gate_act"], T, d)
        ref = float(torch.tensor(0.9)) * X + 0.5 * v * n
        e = (N.rho_err(d) + 40 * N.U) * (0.5 * v * n).abs() + 4 * N.U * (X.abs() + ref.abs())
        N.close(rout, ref, e, f"r{i + 1}")
    ref, _ = N.norm(N.d64(r1), N.d64(w["next0"]), 1e-6)
    N.close(h1, ref, ref.abs() * (N.rho_err(d) + N.CHAIN * N.U), "h1")
    # the gradients at both ends of the first block: D from dr and dh of the second
    V = N.d64(r1)
    wn = N.d64(w["next0"])
    back, eb = N.norm_back(N.d64(g1["dh"]) * wn, V, N.rho_of(V, 1e-6), 2 * N.U * (N.d64(g1["dh"]) * wn).abs())
    D = N.d64(g1["dr"]) + back
    N.close(g0["dr"], float(torch.tensor(0.9)) * D, eb + 4 * N.U * (D.abs() + back.abs()), "dr")
    X = N.d64(r0)
    back, eb = N.norm_back(N.d64(g0["dh"]) * N.d64(w["in"]), X, N.rho_of(X, 1e-6), 2 * N.U * N.d64(g0["dh"]).abs() * 2)
    ref = back + N.d64(g0["dr"])
    N.close(dr, ref, eb + 4 * N.U * (ref.abs() + back.abs()), "dr of the stream")
    t = N.d64(g0["dh"]) * X * N.rho_of(X, 1e-6)
    s, es = N.column(t, t.abs() * (N.rho_err(d) + N.CHAIN * N.U), T)
    N.close(dw_in, s, es, "dw_in")
    # the bias moves, the load is cleared
    before = bias.clone()
    ops.balance_bias(load, bias, 0.01, out=bias)
    assert int(load.sum()) == 0 and float((bias - before).abs().max()) <= 0.0101


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
def test_train_plan_with_scoring(score, renorm):
    """The routed experts on one GPU's share: route, combine with those weights, gate gradient."""
    T, d, f, E, L, k, e0 = 140, 256, 256, 32, 8, 4, 8
    sc = ops.Scoring(score, renorm=renorm, scale=1.5)
    a = inputs(T, d, f, E, 128)
    logits = normal((T, E), 60, 1.5, F32)
    W13, W2 = a["W13"][:L].contiguous(), a["W2"][:L].contiguous()
    p = TrainPlan(T, d, f, E, L, k, e0=e0, device=DEV, scoring=sc)
    wts = quantize_weights(W13, W2, transpose=p.transpose_weights)
    y = p.forward(a["x"], logits, wts)
    l, s, ids = check_route(p, logits, sc, None)
    pr, Y, w = npi(p.pair_row), np64(p.Y), np64(p.w)
    ref = np.where(pr[:, :, None] >= 0, w[:, :, None] * Y[np.maximum(pr, 0)], 0.0)
    tol = U16 * np.abs(ref.sum(1)) + 2 * k * 2.0 ** -24 * np.abs(ref).sum(1) + 1e-30
    close(y, ref.sum(1), tol * 1.01, "y")
    p.backward(a["x"], a["dy"], wts, logits=logits)
    check_route_back(p, l, s, ids, sc)
    with pytest.raises(ValueError):
        p.backward(a["x"], a["dy"], wts)


def test_replayed_step_equals_the_recorded_one():
    """Inference records the scored choice; the trainer's plan replays it: ids, weights and y, bit for bit."""
    T, d, f, E, k = 150, 128, 256, 64, 6
    sc = ops.Scoring("sigmoid", groups=8, top_groups=3, group_top=1, scale=2.0)
    a = inputs(T, d, f, E, 128)
    logits = normal((T, E), 61, 1.5, F32)
    bias = torch.linspace(-0.2, 0.2, E, device=DEV)
    rec = torch.full((3, k, T + 40), -1, dtype=torch.int32, device=DEV)
    ids, w = ops.route_scored(logits, k, sc, bias=bias, capture=(rec, 1, 17))
    wts = quantize_weights(a["W13"], a["W2"])
    p, q = (ForwardPlan(T, d, f, E, E, k, device=DEV, scoring=sc) for _ in range(2))
    p.route_bias = bias
    y = p.forward(a["x"], logits, wts)
    yr = q.forward(a["x"], logits, wts, replay=(rec, 1, 17))
    assert torch.equal(q.ids, ids) and torch.equal(q.w, w) and torch.equal(p.w, w) and torch.equal(y, yr)
    assert int(q.status.item()) == 0
    rec[1, 0, 17 + 3] = E
    q.forward(a["x"], logits, wts, replay=(rec, 1, 17))
    assert int(q.status.item()) == ops.FLAG_BAD_ID and int((q.w[3] != 0).sum()) == 0


def test_block_graph():
    """A block's whole step captured and replayed on new inputs, eager steps between."""
    T, d, f, E, k, fs = 160, 256, 256, 16, 4, 256
    sc = ops.Scoring("softmax", renorm=False)
    a = inputs(T, d, f, E, fs)
    p = MoEBlockPlan(T, d, f, E, k, fs, scoring=sc, device=DEV, gate="full")
    wts = quantize_weights(a["W13"], a["W2"], transpose=p.layer.routed.transpose_weights)
    r, h, d_r, d_h, gate = (normal((T, d), 90 + i) for i in range(5))
    wn = normal((d,), 96, 0.2)

    def step():
        p.forward(r, h, a["Wr"], wts, a["W13s"], a["W2s"], gate=gate, w_next=wn)
        g = p.backward(d_r, d_h, h, a["Wr"], wts, a["W13s"], a["W2s"], gate=gate, w_next=wn)
        return [p.join.r_out, p.join.h] + [t for t in g.values() if t is not None]
    graph = capture_graph(step)
    outs = step()
    for i in range(3):
        h.copy_(normal((T, d), 130 + i))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for s, t in zip(want, outs):
            assert torch.equal(s, t)
