"""The norms around the layer on the GPU against plain 64-bit forms, element by
element within the bounds norm_ref derives."""

import pytest
import torch

import norm_ref as R
from gpu_util import DEV, say
from moe_expert_layer_r3_amd import ops
from moe_expert_layer_r3_amd.block import JoinPlan, NormPlan

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
T_OF = {"bf16": BF, "f32": F32}
EPS = 1e-6


def normal(shape, seed, std=1.0, dtype=BF, mean=0.0, pad=0, rows=False):
    """Seeded values; pad: a column slice of a wider buffer; rows: of very different size."""
    g = torch.Generator().manual_seed(seed)
    if len(shape) == 1:
        return (torch.randn(shape, generator=g) * std + mean).to(dtype).to(DEV)
    t = torch.randn((shape[0], shape[1] + pad), generator=g) * std + mean
    if rows:
        t = t * torch.exp(torch.randn((shape[0], 1), generator=g))
    return t.to(dtype).to(DEV)[:, :shape[1]]


def check_norm(T, d, x_type="bf16", w_type="bf16", pad=0, add=False, train=True, eps=EPS, x=None):
    say(f"norm T={T} d={d} x={x_type} w={w_type} pad={pad} add={add}")
    xt, wt = T_OF[x_type], T_OF[w_type]
    x = normal((T, d), 1, 2.0, xt, pad=pad, rows=True) if x is None else x
    w = normal((d,), 2, 0.3, wt, 1.0)
    p = NormPlan(T, d, x_dtype=xt, w_dtype=wt, eps=eps, train=train, device=DEV)
    h = p.forward(x, w)
    X, W = R.d64(x), R.d64(w)
    ref, rho = R.norm(X, W, eps)
    R.close(h, ref, ref.abs() * (R.rho_err(d) + R.CHAIN * R.U), "h")
    if not train:
        return
    dh = normal((T, d), 3)
    da = normal((T, d), 4, dtype=xt) if add else None
    dx, dw = p.backward(dh, x, w, dx_add=da)
    a = R.d64(dh) * W
    g, e = R.norm_back(a, X, rho, a.abs() * 2 * R.U)
    if add:
        g = g + R.d64(da)
        e = e + 2 * R.U * (g.abs() + R.d64(da).abs())
    R.close(dx, g, e, "dx")
    t = R.d64(dh) * X * rho
    s, es = R.column(t, t.abs() * (R.rho_err(d) + R.CHAIN * R.U), T)
    R.close(dw, s, es, "dw")


NORM_SIZES = [(1, 8), (1, 7168), (3, 64), (7, 128), (130, 520), (5, 512), (66, 1032), (37, 2048), (300, 96), (19, 4104),
              (21, 7168), (9, 8192), (6, 8200), (5, 16384), (3, 16392), (2, 40000), (1025, 256), (700, 24)]


@pytest.mark.parametrize("T,d", NORM_SIZES)
@pytest.mark.parametrize("x_type,w_type", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_norm(T, d, x_type, w_type):
    check_norm(T, d, x_type, w_type, pad=8 * (T % 3), add=d % 16 == 0)


def test_norm_special_rows():
    """Rows of zeros, of subnormal and of large values, and one NaN or infinity that stays in its row."""
    T, d = 12, 640
    x = normal((T, d), 5, dtype=F32)
    x[0] = 0.0
    x[1] = 1e-42
    x[2] *= 1e17
    x[3] *= 1e-12
    check_norm(T, d, "f32", "f32", x=x, eps=1e-6)
    check_norm(T, d, "bf16", "f32", x=x.to(BF), eps=1e-12)
    clean = NormPlan(T, d, x_dtype=F32, train=True, device=DEV)
    w = normal((d,), 2, 0.3, BF, 1.0)
    ref = clean.forward(x, w).clone()
    y = x.clone()
    y[5, 17], y[7, 3] = float("nan"), float("inf")
    h = clean.forward(y, w)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[5] = keep[7] = False
    assert torch.equal(h[keep], ref[keep]) and bool(h[5].isnan().all())


def check_join(T, d, r_type="bf16", w_type="bf16", post=True, pre=True, gate="none", gate_type="bf16", act="none",
               r_scale=1.0, y_scale=1.0, pad=0, with_d_out=True, seed=0, far=False):
    say(f"join T={T} d={d} r={r_type} w={w_type} post={post} pre={pre} gate={gate} {gate_type} {act} scales={r_scale},{y_scale} "
        f"pad={pad} d_out={with_d_out} far={far}")
    rt, wt, gt = T_OF[r_type], T_OF[w_type], T_OF[gate_type]
    y = normal((T, d), 11 + seed, 0.7, pad=pad, rows=True)
    r = normal((T, d), 12 + seed, 2.0, rt, pad=pad, rows=True)
    wp = normal((d,), 13, 0.3, wt, 1.0) if post else None
    wn = normal((d,), 14, 0.3, wt, 1.0) if pre else None
    shape = dict(none=None, channel=(d,), token=(T,), full=(T, d))[gate]
    gv = None if shape is None else normal(shape, 15, 0.8, gt, 0.2).contiguous()
    if far:
        gv.view(-1)[:len(FAR)] = torch.tensor(FAR, device=DEV).to(gt)[:gv.numel()]
    p = JoinPlan(T, d, r_dtype=rt, w_dtype=wt, post=post, pre=pre, gate=gate, gate_dtype=gt, gate_act=act, r_scale=r_scale,
                 y_scale=y_scale, eps=EPS, train=True, device=DEV)
    r_out, h = p.forward(y, r, w_post=wp, gate=gv, w_pre=wn)
    rs, ys = float(torch.tensor(r_scale)), float(torch.tensor(y_scale))
    Y, X = R.d64(y), R.d64(r)
    re, u = R.rho_err(d), R.U
    if post:
        n, rho_y = R.norm(Y, R.d64(wp), EPS)
        en = n.abs() * (re + R.CHAIN * u)
    else:
        n, en, rho_y = Y, 0 * Y, torch.ones(1, 1, dtype=torch.float64)
    g, slope = R.gate_of(gv, gate, act, T, d)
    # exp, a sum and a division; 0 without an activation. Below the normal range a gate and its slope may be 0
    tiny = 2.0 ** -126 if far else 0.0
    eg = 8 * u * g.abs() + tiny
    z, ez = g * n, g.abs() * en + eg * (n.abs() + en)
    ref = rs * X + ys * z
    R.close(r_out, ref, abs(ys) * ez + 3 * u * ((rs * X).abs() + (ys * z).abs()), "r_out")
    V = R.d64(r_out)                   # the stream goes on as it is stored
    if pre:
        hn, rho = R.norm(V, R.d64(wn), EPS)
        R.close(h, hn, hn.abs() * (re + R.CHAIN * u), "h")
    else:
        assert h is None
    d_out = normal((T, d), 16, dtype=rt) if with_d_out else None
    dh = normal((T, d), 17) if pre else None
    got = p.backward(d_out, dh, y, w_post=wp, gate=gv, w_pre=wn)
    D = torch.zeros(T, d, dtype=torch.float64) if d_out is None else R.d64(d_out)
    eD = 0 * D
    if pre:
        a = R.d64(dh) * R.d64(wn)
        b, eb = R.norm_back(a, V, rho, 2 * u * a.abs())
        D, eD = D + b, eb + 2 * u * (D.abs() + b.abs())
        t = R.d64(dh) * V * rho
        s, es = R.column(t, t.abs() * (re + R.CHAIN * u), T)
        R.close(got["dw_pre"], s, es, "dw_pre")
    R.close(got["dr"], rs * D, abs(rs) * eD + u * (rs * D).abs(), "dr")
    dz, edz = ys * D, abs(ys) * eD + u * (ys * D).abs()
    if gate != "none":
        t, et = dz * n * slope, (edz * (n.abs() + en) + dz.abs() * en + 20 * u * (dz * n).abs()) * slope.abs() + tiny * (dz * n).abs()
        if gate == "channel":
            t, et = R.column(t, et, T)
        elif gate == "token":
            et = et.sum(dim=1) + (d + 16) * u * (t.abs() + et).sum(dim=1)
            t = t.sum(dim=1)
        R.close(got["dgate"], t, et, "dgate")
    dn, edn = dz * g, edz * g.abs() + eg * (dz.abs() + edz) + u * (dz * g).abs()
    if post:
        t = dn * Y * rho_y
        s, es = R.column(t, edn * (Y * rho_y).abs() * (1 + re) + t.abs() * (re + R.CHAIN * u), T)
        R.close(got["dw_post"], s, es, "dw_post")
        w = R.d64(wp)
        dn, edn = R.norm_back(dn * w, Y, rho_y, (edn + 2 * u * dn.abs()) * w.abs())
    R.close(got["dy"], dn, edn, "dy")
    return p, (y, r, wp, gv, wn, d_out, dh)


@pytest.mark.parametrize("gate,act", [("none", "none"), ("channel", "none"), ("channel", "sigmoid"), ("token", "sigmoid"),
                                      ("token", "none"), ("full", "sigmoid"), ("full", "none")])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("bf16", "f32", "bf16"),
                                   ("f32", "bf16", "f32")])
def test_join_forms(gate, act, post, pre, types):
    check_join(45, 264, *types[:2], post, pre, gate, types[2], act, 0.75, 0.5, pad=8)
    check_join(6, 1544, *types[:2], post, pre, gate, types[2], act, 1.0, -2.0)
    check_join(5, 10008, *types[:2], post, pre, gate, types[2], act, 1.0, 0.5, pad=16)


@pytest.mark.parametrize("T,d", NORM_SIZES)
@pytest.mark.parametrize("gate,r_type", [("channel", "bf16"), ("full", "f32"), ("token", "f32")])
def test_join_sizes(T, d, gate, r_type):
    check_join(T, d, r_type, "bf16" if d % 3 else "f32", gate=gate, act="sigmoid", gate_type="f32" if d % 5 else "bf16",
               r_scale=0.5, y_scale=1.5, pad=16 * (T % 2), with_d_out=T % 4 != 1)


# gates far out, where the exponential leaves its range on either side
FAR = [float("inf"), -float("inf"), 3e38, -3e38, 1e30, -1e30, 129.0, -129.0, 104.0, -104.0, 90.0, -90.0, 87.0, -87.0, 50.0, -50.0,
       0.0, -0.0]


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
@pytest.mark.parametrize("T,d", [(45, 264), (40, 5000), (21, 8200), (18, 16400)])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")])
def test_join_far_gates(gate, T, d, types):
    """Sigmoid gates up to infinity: 0 or 1, without a slope."""
    p, (_, _, _, gv, *_) = check_join(T, d, types[0], gate=gate, gate_type=types[1], act="sigmoid", far=True)
    assert bool(p.dgate.isfinite().all()) and bool((p.dgate.view(-1)[:8] == 0).all())
    assert all(bool(t.isfinite().all()) for t in (p.r_out, p.h, p.dr, p.dy, p.dw_post, p.dw_pre))


def test_many_rows():
    """More rows than workgroups: every partial sum, the tails, and unequal shares of rows."""
    for T, d in ((4099, 64), (1500, 1032), (1027, 7168), (600, 12296)):
        check_join(T, d, gate="channel", act="sigmoid", y_scale=0.5)
        check_norm(T, d, "f32", "f32", add=True)


def test_gradient_against_differences():
    """Gradients of the 64-bit forms (which the kernels' tests use) against central differences, and the kernel's
    own against them, at a small size."""
    T, d = 3, 16
    p, (y, r, wp, gv, wn, d_out, dh) = check_join(T, d, "f32", "f32", gate="full", gate_type="f32", act="sigmoid",
                                                  r_scale=0.75, y_scale=0.5)
    got = p.backward(d_out, dh, y, w_post=wp, gate=gv, w_pre=wn)
    v = dict(y=R.d64(y), r=R.d64(r), wp=R.d64(wp), g=R.d64(gv), wn=R.d64(wn))
    A, B = R.d64(d_out), R.d64(dh)

    def loss(v):
        n, _ = R.norm(v["y"], v["wp"], EPS)
        out = 0.75 * v["r"] + 0.5 * torch.sigmoid(v["g"]) * n
        return float((A * out).sum() + (B * R.norm(out, v["wn"], EPS)[0]).sum())
    step = 1e-5
    for name, grad in (("y", "dy"), ("r", "dr"), ("wp", "dw_post"), ("g", "dgate"), ("wn", "dw_pre")):
        flat, g = v[name].flatten(), R.d64(got[grad]).flatten()
        scale = float(g.abs().max())
        for i in range(flat.numel()):
            keep = float(flat[i])
            vals = []
            for s in (step, -step):
                flat[i] = keep + s
                vals.append(loss({**v, name: flat.view(v[name].shape)}))
            flat[i] = keep
            diff = (vals[0] - vals[1]) / (2 * step)
            # bf16 gradients: half a step; the rest: the stored stream and differences, far below 1e-5 of the largest
            tol = (2.0 ** -8 if got[grad].dtype == BF else 0.0) * abs(diff) + 1e-5 * scale
            assert abs(float(g[i]) - diff) <= tol, (name, i, float(g[i]), diff)


def test_in_place_and_untouched():
    """r_out over r, dr over d_out, dx over dx_add; nothing written past an output or in the columns beside a slice."""
    T, d, pad = 33, 520, 24
    y, r = normal((T, d), 1), normal((T, d), 2, dtype=F32)
    wp, wn = normal((d,), 3, 0.3, BF, 1.0), normal((d,), 4, 0.3, BF, 1.0)
    p = JoinPlan(T, d, r_dtype=F32, train=True, device=DEV)
    r_out, h = p.forward(y, r, w_post=wp, w_pre=wn)
    guard = torch.full((T * d + 64,), 7.0, device=DEV)
    over = guard[:T * d].view(T, d)
    over.copy_(r)
    h2 = torch.full((T * d + 64,), 7.0, dtype=BF, device=DEV)
    st = torch.full((2, T + 16), 7.0, device=DEV)
    ops.launch("moe_join", y.device, y.data_ptr(), d, over.data_ptr(), 1, d, wp.data_ptr(), None, 0, 0, 0, 1.0, 1.0,
               wn.data_ptr(), 0, T, d, 1e-6, over.data_ptr(), h2.data_ptr(), st[0].data_ptr(), st[1].data_ptr())
    assert torch.equal(over, r_out) and torch.equal(h2[:T * d].view(T, d), h)
    assert bool((guard[T * d:] == 7).all()) and bool((h2[T * d:] == 7).all()) and bool((st[:, T:] == 7).all())
    d_out, dh = normal((T, d), 5, dtype=F32), normal((T, d), 6)
    want = {k: v.clone() for k, v in p.backward(d_out, dh, y, w_post=wp, w_pre=wn).items() if v is not None}
    dy2 = torch.full((T * d + 64,), 7.0, dtype=BF, device=DEV)
    dw = torch.full((2, d + 64), 7.0, dtype=BF, device=DEV)
    ws = torch.empty_like(p.ws)
    ops.launch("moe_join_backward", y.device, d_out.data_ptr(), dh.data_ptr(), y.data_ptr(), d, r_out.data_ptr(), 1,
               wp.data_ptr(), None, 0, 0, 0, 1.0, 1.0, wn.data_ptr(), 0, st[0].data_ptr(), st[1].data_ptr(), T, d,
               d_out.data_ptr(), dy2.data_ptr(), dw[0].data_ptr(), dw[1].data_ptr(), None, ws.data_ptr(), ws.numel())
    assert torch.equal(d_out, want["dr"]) and torch.equal(dy2[:T * d].view(T, d), want["dy"])
    assert torch.equal(dw[0, :d], want["dw_post"]) and torch.equal(dw[1, :d], want["dw_pre"])
    assert bool((dy2[T * d:] == 7).all()) and bool((dw[:, d:] == 7).all())
    q = NormPlan(T, d, x_dtype=F32, train=True, device=DEV)
    q.forward(r, wn)
    add = normal((T, d), 8, dtype=F32)
    dx, dwn = (t.clone() for t in q.backward(dh, r, wn, dx_add=add))
    ops.launch("moe_norm_backward", y.device, dh.data_ptr(), r.data_ptr(), 1, d, wn.data_ptr(), 0, q.rstd.data_ptr(),
               add.data_ptr(), T, d, add.data_ptr(), None, q.ws.data_ptr(), q.ws.numel())
    assert torch.equal(add, dx)
    wide = normal((T, d + pad), 9)
    keep = wide.clone()
    NormPlan(T, d, device=DEV).forward(wide[:, :d], wn)
    assert torch.equal(wide, keep)


def test_each_gradient_alone():
    """Any one gradient asked for is the one that all together give."""
    T, d = 70, 264
    p, (y, r, wp, gv, wn, d_out, dh) = check_join(T, d, gate="channel", act="sigmoid")
    want = p.backward(d_out, dh, y, w_post=wp, gate=gv, w_pre=wn)
    names = ("dr", "dy", "dw_post", "dw_pre", "dgate")
    for one in names:
        outs = [torch.full_like(want[n], 3.0) for n in names]
        ops.launch("moe_join_backward", y.device, d_out.data_ptr(), dh.data_ptr(), y.data_ptr(), d, p.r_out.data_ptr(), 0,
                   wp.data_ptr(), gv.data_ptr(), *p.gate_args, wn.data_ptr(), 0, p.rstd_post.data_ptr(),
                   p.rstd_pre.data_ptr(), T, d, *[o.data_ptr() if n == one else None for o, n in zip(outs, names)],
                   p.ws.data_ptr(), p.ws.numel())
        for o, n in zip(outs, names):
            assert torch.equal(o, want[n]) if n == one else bool((o == 3).all()), (one, n)


def test_empty_batch():
    d = 64
    p = JoinPlan(0, d, gate="channel", train=True, device=DEV)
    z = lambda dt=BF: torch.empty((0, d), dtype=dt, device=DEV)
    w, g = normal((d,), 1), normal((d,), 2)
    p.forward(z(), z(), w_post=w, gate=g, w_pre=w)
    for t in (p.dw_post, p.dw_pre, p.dgate):
        t.fill_(5.0)
    got = p.backward(z(), z(), z(), w_post=w, gate=g, w_pre=w)
    assert all(int((got[n] != 0).sum()) == 0 for n in ("dw_post", "dw_pre", "dgate"))
    q = NormPlan(0, d, train=True, device=DEV)
    q.forward(z(), w)
    q.dw.fill_(5.0)
    assert int((q.backward(z(), z(), w)[1] != 0).sum()) == 0


def test_refusals_of_plans():
    T, d = 4, 64
    p = JoinPlan(T, d, device=DEV)
    y, w = normal((T, d), 1), normal((d,), 2)
    for kw in (dict(w_post=w), dict(w_pre=w), dict(w_post=w, w_pre=w, gate=w), dict(w_post=w.float(), w_pre=w),
               dict(w_post=w[:32], w_pre=w)):
        with pytest.raises(ValueError):
            p.forward(y, y, **kw)
    with pytest.raises(TypeError):
        p.forward(y, y.float(), w_post=w, w_pre=w)
    with pytest.raises(ValueError):
        p.forward(y, y[:, ::2], w_post=w, w_pre=w)
    with pytest.raises(ValueError):
        p.backward(y, y, y, w_post=w, w_pre=w)
    with pytest.raises(ops.MoeError):       # rows 12 elements apart
        NormPlan(T, 8, device=DEV).forward(normal((T, 12), 1)[:, :8], w[:8])
    with pytest.raises(ValueError):
        JoinPlan(T, d, gate="row", device=DEV)
    with pytest.raises(ValueError):
        JoinPlan(T, d, gate_act="silu", device=DEV)


def test_graph_and_streams():
    """Forward and backward captured, replayed several times with eager work between; a side stream gives the same."""
    from moe_expert_layer_r3_amd.layer import capture_graph
    T, d = 260, 7168
    p = JoinPlan(T, d, gate="channel", train=True, device=DEV)
    y, r, d_out, dh = (normal((T, d), i) for i in range(4))
    wp, wn, g = (normal((d,), 10 + i, 0.3, BF, 1.0) for i in range(3))

    def step(q):
        q.forward(y, r, w_post=wp, gate=g, w_pre=wn)
        q.backward(d_out, dh, y, w_post=wp, gate=g, w_pre=wn)
        return [q.r_out, q.h, q.dr, q.dy, q.dw_post, q.dw_pre, q.dgate]
    graph = capture_graph(lambda: step(p))
    q = JoinPlan(T, d, gate="channel", train=True, device=DEV)
    for seed in range(3):
        y.copy_(normal((T, d), 100 + seed))
        graph.replay()
        torch.cuda.synchronize()
        want = step(q)
        for a, b in zip([p.r_out, p.h, p.dr, p.dy, p.dw_post, p.dw_pre, p.dgate], want):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = JoinPlan(T, d, gate="channel", train=True, device=DEV)
    with torch.cuda.stream(side):
        got = step(s)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [264, 1032, 7168, 12296])
def test_two_streams_at_once(d):
    """Plans of their own on two streams, calls in flight on both: each gives what it gives alone."""
    T = 900
    y, r, d_out, dh = (normal((T, d), 20 + i) for i in range(4))
    wp, wn, g = (normal((d,), 30 + i, 0.3, BF, 1.0) for i in range(3))
    plans = [JoinPlan(T, d, gate="channel", gate_act=act, train=True, device=DEV) for act in ("none", "sigmoid")]

    def step(p):
        p.forward(y, r, w_post=wp, gate=g, w_pre=wn)
        p.backward(d_out, dh, y, w_post=wp, gate=g, w_pre=wn)
        return p.r_out, p.h, p.dr, p.dy, p.dw_post, p.dw_pre, p.dgate
    want = [[t.clone() for t in step(p)] for p in plans]
    sides = [torch.cuda.Stream() for _ in plans]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for p, s in zip(plans, sides):
            with torch.cuda.stream(s):
                step(p)
    for s in sides:
        s.synchronize()
    for p, w in zip(plans, want):
        for a, b in zip((p.r_out, p.h, p.dr, p.dy, p.dw_post, p.dw_pre, p.dgate), w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,d", [(40, 264), (12, 5000), (5, 8200), (4, 16400)])
@pytest.mark.parametrize("act", ["none", "sigmoid"])
def test_nan_gate_stays_in_its_row(T, d, act):
    """A gate of NaN makes its own row NaN, forward and back, and no other."""
    y, r, d_out, dh, g = (normal((T, d), 40 + i) for i in range(5))
    wp, wn = (normal((d,), 50 + i, 0.3, BF, 1.0) for i in range(2))
    p = JoinPlan(T, d, gate="full", gate_act=act, train=True, device=DEV)

    def step():
        p.forward(y, r, w_post=wp, gate=g, w_pre=wn)
        p.backward(d_out, dh, y, w_post=wp, gate=g, w_pre=wn)
        return [t.clone() for t in (p.r_out, p.h, p.dr, p.dy, p.dgate)]
    want = step()
    g[2, 17] = float("nan")
    got = step()
    keep = torch.arange(T, device=DEV) != 2
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep])
    assert bool(got[0][2, 17].isnan()) and all(bool(t[2].isnan().all()) for t in got[1:4])
