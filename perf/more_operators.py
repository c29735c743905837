"""Cases and plain forms of the operators at a layer's borders.

Two things stand between a model's residual stream and the experts of a
Mixture-of-Experts layer:
  route    the choice of experts by scores: softmax or sigmoid scores of the
           router's logits, a bias per expert that only the choice sees, groups of
           experts of which the best stay, top-k, weights that are renormalised or
           not; its gradient; the update of the bias from the experts' load; the
           choice written into a record
  replay   the same weights for experts that a record names, and their gradient
  norm     the root-mean-square norm in front of the layer, and its gradients
  join     what follows it, in one pass: the norm of the layer's output y, a gate,
           the residual scale and sum, and the next layer's norm,
             r' = r_scale r + y_scale g n(y),  h = norm(r')
           and the gradients of all of it

Scores are values of 32 bits, rounded once from the function's value; where two are
equal the lower index wins.

``own`` chooses between the framework's kernels and elementary torch operations.
"""

import math

import torch

own = False

DEV = "cuda:0"
BF = torch.bfloat16
F32 = torch.float32
TYPES = {"bf16": BF, "f32": F32}
EPS = 1e-6


def _route(name, T, E, k, score, bias=False, groups=1, top_groups=1, group_top=2, renorm=True, scale=1.0, logits="f32",
           masked=False, capture=False, train=False, balance=False):
    return dict(name=name, kind="route", T=T, E=E, k=k, score=score, bias=bias, groups=groups, top_groups=top_groups,
                group_top=group_top, renorm=renorm, scale=scale, logits=logits, masked=masked, capture=capture,
                train=train, balance=balance)


def _replay(name, T, E, k, score, renorm=True, scale=1.0, logits="f32", train=False):
    return dict(name=name, kind="replay", T=T, E=E, k=k, score=score, renorm=renorm, scale=scale, logits=logits,
                train=train)


def _norm(name, T, d, x="bf16", w="bf16", pad=0, add=False, train=False):
    return dict(name=name, kind="norm", T=T, d=d, x=x, w=w, pad=pad, add=add, train=train)


def _join(name, T, d, r="bf16", w="bf16", post=True, pre=True, gate="none", gate_type="bf16", act="none", r_scale=1.0,
          y_scale=1.0, pad=0, train=False):
    return dict(name=name, kind="join", T=T, d=d, r=r, w=w, post=post, pre=pre, gate=gate, gate_type=gate_type, act=act,
                r_scale=r_scale, y_scale=y_scale, pad=pad, train=train)


def listed():
    return [
        # one decoded token: sigmoid scores, the best 4 of 8 groups, the balance bias
        _route("route_token", 1, 256, 8, "sigmoid", bias=True, groups=8, top_groups=4, scale=2.5),
        # a small training batch of a router with odd sizes: softmax over bf16 logits, masked experts, groups by their best
        _route("route_ragged", 1237, 60, 6, "softmax", groups=5, top_groups=2, group_top=1, renorm=False, logits="bf16",
               masked=True, train=True),
        # a training step's router: choice, gradient, and the bias moved towards even load
        _route("route_train", 16384, 256, 8, "sigmoid", bias=True, groups=8, top_groups=4, scale=2.5, train=True,
               balance=True),
        # inference over a whole recorded sequence: the choice is written into one layer of the record
        _route("route_long", 131072, 256, 8, "sigmoid", bias=True, groups=8, top_groups=4, scale=2.5, capture=True),
        # one chunk of a recorded sequence replayed
        _replay("replay_chunk", 16384, 256, 8, "sigmoid", scale=2.5),
        # the same in a training step, with softmax scores that are not renormalised: every logit has a gradient
        _replay("replay_train", 16384, 256, 8, "softmax", renorm=False, train=True),
        # the norm in front of the layer for one decoded token
        _norm("norm_token", 1, 7168),
        # the same in a training step, with the residual stream kept in 32 bits
        _norm("norm_train", 16384, 7168, x="f32", w="f32", add=True, train=True),
        # a decode batch behind a layer: a gate per token, residual stream in 32 bits
        _join("join_batch", 48, 7168, r="f32", gate="token", gate_type="f32", act="sigmoid"),
        # prompt tokens: norm behind the layer, scaled residual sum, norm of the next layer
        _join("join_prompt", 16384, 7168, r_scale=0.75, y_scale=0.5),
        # a training step at the border of two layers: a gate per channel
        _join("join_train", 16384, 7168, gate="channel", y_scale=0.5, train=True),
        # a small training batch with odd sizes and an element-wise gate, from a column slice of a wider buffer
        _join("join_ragged", 1237, 1032, r="f32", w="f32", gate="full", act="sigmoid", r_scale=0.75, pad=24, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "route", "route", "replay", "norm", "join", "join"])
    if kind in ("route", "replay"):
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512, _log(rng, 8, 1024)])
        T = min(_log(rng, 1, 131072), 131072 * 256 // E)
        k = rng.randint(1, min(16, E)) if rng.random() < 0.5 else min(8, E)
        score, renorm = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6
        scale, logits = rng.choice([1.0, 2.5]), rng.choice(["f32", "f32", "bf16"])
        train = rng.random() < 0.5
        if kind == "replay":
            c = _replay("", T, E, k, score, renorm, scale, logits, train)
        else:
            G = rng.choice([g for g in range(1, 33) if E % g == 0 and E // g >= 2] or [1])
            G = 1 if rng.random() < 0.3 else G
            H = rng.randint(-(-k * G // E), G)
            c = _route("", T, E, k, score, rng.random() < 0.6, G, H, rng.choice([1, 2]) if E // G >= 2 else 1, renorm, scale,
                       logits, rng.random() < 0.2, rng.random() < 0.25, train, rng.random() < 0.3)
            c["balance"] = c["balance"] and c["bias"]
    elif kind == "norm":
        d = 8 * _log(rng, 8, 1024)
        c = _norm("", min(_log(rng, 1, 131072), 16384 * 7168 // d), d, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]),
                  8 * rng.choice([0, 0, 1, 5]), rng.random() < 0.5, rng.random() < 0.6)
    else:
        d = 8 * _log(rng, 8, 1024)
        post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        gate = rng.choice(["none", "channel", "token", "full"])
        c = _join("", min(_log(rng, 1, 131072), 16384 * 7168 // d // 2), d, rng.choice(["bf16", "f32"]),
                  rng.choice(["bf16", "f32"]), post, pre, gate, rng.choice(["bf16", "f32"]),
                  rng.choice(["none", "sigmoid"]) if gate != "none" else "none", rng.choice([1.0, 0.75]),
                  rng.choice([1.0, 0.5]), 8 * rng.choice([0, 0, 1, 5]), rng.random() < 0.6)
    del c["name"]
    return c


# ------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(shape, std=1.0, dtype=BF, mean=0.0):
        return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(dtype)

    st, T = dict(case=case), case["T"]
    if case["kind"] in ("route", "replay"):
        E, k = case["E"], case["k"]
        # some experts are liked more than others, as a router in training has it
        lean = torch.randn(E, generator=g, device=DEV) * 0.5
        logits = torch.randn((T, E), generator=g, device=DEV) * 1.2 + lean
        if case.get("masked"):
            off = torch.rand((T, E), generator=g, device=DEV) < 0.1
            logits = torch.where(off, torch.full_like(logits, -math.inf), logits)
        st["logits"] = logits.to(TYPES[case["logits"]])
        if case["kind"] == "replay":
            S = T + 1000
            st["s0"] = 500
            rec = torch.rand((S, E), generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
            st["rec"] = torch.stack([rec.t().contiguous().roll(1, 1), rec.t().contiguous()]).contiguous()
        else:
            st["bias"] = torch.randn(E, generator=g, device=DEV) * 0.05 - lean * 0.1 if case["bias"] else None
            if case["capture"]:
                st["rec"] = torch.full((4, k, T + 77), -1, dtype=torch.int32, device=DEV)
            if case["balance"]:
                st["load"] = torch.zeros(E, dtype=torch.int32, device=DEV)
        if case["train"]:
            st["d_w"] = normal((T, k), 1.0, F32)
        if own:
            from moe_expert_layer_r3_amd import ops
            from moe_expert_layer_r3_amd.block import RoutePlan
            sc = ops.Scoring(case["score"], groups=case.get("groups", 1), top_groups=case.get("top_groups", 1),
                             group_top=case.get("group_top", 2), renorm=case["renorm"], scale=case["scale"])
            st["plan"] = RoutePlan(T, E, k, sc, logits_dtype=TYPES[case["logits"]], train=case["train"], device=DEV)
        return st
    d, pad, wt = case["d"], case["pad"], TYPES[case["w"]]
    # rows of very different size, as residual streams have them
    size = torch.exp(torch.randn((T, 1), generator=g, device=DEV) * 0.7 + 1.0)
    if case["kind"] == "norm":
        xt = TYPES[case["x"]]
        st["x"] = (torch.randn((T, d + pad), generator=g, device=DEV) * size).to(xt)[:, :d]
        st["w"] = normal((d,), 0.2, wt, 1.0)
        if case["train"]:
            st["dh"] = normal((T, d))
            st["add"] = normal((T, d), 1.0, xt) if case["add"] else None
        if own:
            from moe_expert_layer_r3_amd.block import NormPlan
            st["plan"] = NormPlan(T, d, x_dtype=xt, w_dtype=wt, eps=EPS, train=case["train"], device=DEV)
        return st
    rt = TYPES[case["r"]]
    st["r"] = (torch.randn((T, d + pad), generator=g, device=DEV) * size).to(rt)[:, :d]
    st["y"] = (torch.randn((T, d + pad), generator=g, device=DEV) * size * 0.3).to(BF)[:, :d]
    st["w_post"] = normal((d,), 0.2, wt, 1.0) if case["post"] else None
    st["w_pre"] = normal((d,), 0.2, wt, 1.0) if case["pre"] else None
    shape = dict(none=None, channel=(d,), token=(T,), full=(T, d))[case["gate"]]
    st["gate"] = None if shape is None else normal(shape, 0.7, TYPES[case["gate_type"]], 0.3)
    if case["train"]:
        st["d_out"] = normal((T, d), 1.0, rt)
        st["dh"] = normal((T, d)) if case["pre"] else None
    if own:
        from moe_expert_layer_r3_amd.block import JoinPlan
        st["plan"] = JoinPlan(T, d, r_dtype=rt, w_dtype=wt, post=case["post"], pre=case["pre"], gate=case["gate"],
                              gate_dtype=TYPES[case["gate_type"]], gate_act=case["act"], r_scale=case["r_scale"],
                              y_scale=case["y_scale"], eps=EPS, train=case["train"], device=DEV)
    return st


def run(state):
    kind = state["case"]["kind"]
    if own:
        return dict(route=_own_route, replay=_own_route, norm=_own_norm, join=_own_join)[kind](state)
    return dict(route=_plain_route, replay=_plain_route, norm=_plain_norm, join=_plain_join)[kind](state)


# ------------------------------------------------------------ the framework

STEP = 0.001  # of the balance bias


def _own_route(st):
    c, p = st["case"], st["plan"]
    out = {}
    if c["kind"] == "replay":
        out["ids"], out["w"] = p.replay(st["rec"], 1, st["s0"], st["logits"])
    else:
        out["ids"], out["w"] = p.forward(st["logits"], bias=st["bias"], load=st.get("load"),
                                         capture=(st["rec"], 2, 50) if c["capture"] else None)
        if c["capture"]:
            out["rec"] = st["rec"]
        if c["balance"]:
            from moe_expert_layer_r3_amd import ops
            out["bias"] = ops.balance_bias(st["load"], st["bias"], STEP)
    if c["train"]:
        out["d_logits"] = p.backward(st["d_w"], st["logits"])
    return out


def _own_norm(st):
    p = st["plan"]
    out = dict(h=p.forward(st["x"], st["w"]))
    if st["case"]["train"]:
        out["dx"], out["dw"] = p.backward(st["dh"], st["x"], st["w"], dx_add=st["add"])
    return out


def _own_join(st):
    p, c = st["plan"], st["case"]
    out = {}
    out["r"], h = p.forward(st["y"], st["r"], w_post=st["w_post"], gate=st["gate"], w_pre=st["w_pre"])
    if c["pre"]:
        out["h"] = h
    if c["train"]:
        g = p.backward(st["d_out"], st["dh"], st["y"], w_post=st["w_post"], gate=st["gate"], w_pre=st["w_pre"])
        out.update({n: t for n, t in g.items() if t is not None})
    return out


# ------------------------------------------------------------ plain forms

def _scores(c, logits):
    """Scores in 64 bits: they decide between experts where 32 bits would not."""
    # a logit of -inf or of the type's lowest value masks its expert
    l = logits.double()
    l = torch.where(logits <= torch.finfo(logits.dtype).min, torch.full_like(l, -math.inf), l)
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    m = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - m)
    s = e / e.sum(dim=1, keepdim=True)
    return torch.where(m == -math.inf, torch.zeros_like(s), s)


def _plain_choice(c, logits, s32, bias):
    T, E, G = c["T"], c["E"], c["groups"]
    v = s32 if bias is None else s32 + bias
    v = torch.where(logits <= torch.finfo(logits.dtype).min, torch.full_like(v, -math.inf), v)
    if G > 1:
        top = v.view(T, G, E // G).sort(dim=2, descending=True, stable=True).values[:, :, :c["group_top"]]
        value = torch.where(top == -math.inf, torch.zeros_like(top), top).sum(dim=2)
        value = torch.where(top[:, :, 0] == -math.inf, torch.full_like(value, -math.inf), value)
        kept = value.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=v.device)
        keep.scatter_(1, kept, True)
        keep = keep.repeat_interleave(E // G, dim=1)
        # experts of the other groups come after every expert of a kept one, masked ones among them too
        order = v.sort(dim=1, descending=True, stable=True).indices
        first = torch.gather(~keep, 1, order).to(torch.int8).sort(dim=1, stable=True).indices
        return torch.gather(order, 1, first)[:, :c["k"]]
    return v.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]


def _plain_route(st):
    c, logits = st["case"], st["logits"]
    T, E, k = c["T"], c["E"], c["k"]
    s = _scores(c, logits)
    out = {}
    if c["kind"] == "replay":
        ids = st["rec"][1, :, st["s0"]:st["s0"] + T].t().long()
    else:
        ids = _plain_choice(c, logits, s.float(), st["bias"])
        if c["capture"]:
            st["rec"][2, :, 50:50 + T] = ids.t().to(torch.int32)
            out["rec"] = st["rec"]
        if c["balance"]:
            load = torch.zeros(E, dtype=torch.int64, device=DEV)
            load.index_add_(0, ids.reshape(-1), torch.ones(T * k, dtype=torch.int64, device=DEV))
            out["bias"] = st["bias"] + STEP * torch.sign(load.sum() - E * load).float()
    sel = torch.gather(s, 1, ids)
    total = sel.sum(dim=1, keepdim=True)
    share = torch.where(total > 0, sel / total, torch.zeros_like(sel)) if c["renorm"] else sel
    out["ids"] = ids.to(torch.int32)
    out["w"] = (share * c["scale"]).float()
    if c["train"]:
        d_w = st["d_w"].double() * c["scale"]
        if c["renorm"]:
            d = share * (d_w - (d_w * share).sum(dim=1, keepdim=True))   # of the selected scores' logarithms
        else:
            d = sel * d_w
        dl = torch.zeros((T, E), dtype=torch.float64, device=DEV)
        if c["score"] == "sigmoid":
            far = torch.gather(1.0 / (1.0 + torch.exp(logits.double())), 1, ids)
            dl.scatter_add_(1, ids, d * far)
        else:
            dl.scatter_add_(1, ids, d)
            if not c["renorm"]:
                dl -= s * d.sum(dim=1, keepdim=True)
        out["d_logits"] = dl.to(logits.dtype)
    return out


def _rho(v):
    return 1.0 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)


def _norm_back(a, x, rho):
    """Gradient of x * rho for the gradient a."""
    xh = x * rho
    return rho * (a - xh * (a * xh).mean(dim=1, keepdim=True))


def _plain_norm(st):
    c = st["case"]
    x, w = st["x"].float(), st["w"].float()
    rho = _rho(x)
    out = dict(h=(x * rho * w).to(BF))
    if c["train"]:
        dh = st["dh"].float()
        dx = _norm_back(dh * w, x, rho)
        if st["add"] is not None:
            dx = dx + st["add"].float()
        out["dx"] = dx.to(st["x"].dtype)
        out["dw"] = (dh * x * rho).double().sum(dim=0).to(st["w"].dtype)
    return out


def _gate(c, g):
    """(gate, slope) spread over [T, d] or broadcast to it."""
    if g is None:
        return 1.0, None
    g = g.float()
    g = g.view(1, -1) if c["gate"] == "channel" else g.view(-1, 1) if c["gate"] == "token" else g
    if c["act"] == "sigmoid":
        v = 1.0 / (1.0 + torch.exp(-g))
        return v, v / (1.0 + torch.exp(g))
    return g, torch.ones_like(g)


def _plain_join(st):
    c = st["case"]
    y, r = st["y"].float(), st["r"].float()
    n, rho_y = y, None
    if c["post"]:
        rho_y = _rho(y)
        n = y * rho_y * st["w_post"].float()
    g, slope = _gate(c, st["gate"])
    r_out = (c["r_scale"] * r + c["y_scale"] * (g * n)).to(st["r"].dtype)
    out = dict(r=r_out)
    rv = r_out.float()
    if c["pre"]:
        rho = _rho(rv)
        out["h"] = (rv * rho * st["w_pre"].float()).to(BF)
    if not c["train"]:
        return out
    D = st["d_out"].float()
    if c["pre"]:
        dh = st["dh"].float()
        D = D + _norm_back(dh * st["w_pre"].float(), rv, rho)
        out["dw_pre"] = (dh * rv * rho).double().sum(dim=0).to(st["w_pre"].dtype)
    out["dr"] = (c["r_scale"] * D).to(st["r"].dtype)
    dz = c["y_scale"] * D
    if slope is not None:
        dg = dz * n * slope
        if c["gate"] == "channel":
            dg = dg.double().sum(dim=0)
        elif c["gate"] == "token":
            dg = dg.double().sum(dim=1)
        out["dgate"] = dg.to(st["gate"].dtype)
    dn = dz * g
    if c["post"]:
        out["dw_post"] = (dn * y * rho_y).double().sum(dim=0).to(st["w_post"].dtype)
        dn = _norm_back(dn * st["w_post"].float(), y, rho_y)
    out["dy"] = dn.to(BF)
    return out


# ------------------------------------------------------------ what a pass cannot do without

def work(case):
    T = case["T"]
    size = {"bf16": 2, "f32": 4}
    if case["kind"] in ("route", "replay"):
        E, k, o = case["E"], case["k"], size[case["logits"]]
        whole = case["kind"] == "route" or (case["score"] == "softmax" and not case["renorm"])
        b = o * (T * E if whole else T * k) + 8 * T * k   # logits; ids and weights
        b += 4 * T * k if case["kind"] == "replay" or case["capture"] else 0
        if case["train"]:
            b += 4 * T * k + o * T * E
        per = 8 if case["score"] == "sigmoid" else 6
        return dict(bytes=b, flops=T * ((E if whole else k) * per + 4 * k) * (2 if case["train"] else 1))
    d, wt = case["d"], size[case["w"]]
    if case["kind"] == "norm":
        x = size[case["x"]]
        b = T * d * (x + 2) + wt * d
        if case["train"]:
            b += T * d * (2 + x + x + (x if case["add"] else 0)) + wt * d
        return dict(bytes=b, flops=T * d * (4 + (12 if case["train"] else 0)))
    r, norms = size[case["r"]], case["post"] + case["pre"]
    gate = size[case["gate_type"]] * dict(none=0, channel=d, token=T, full=T * d)[case["gate"]]
    b = T * d * (2 + r + r + (2 if case["pre"] else 0)) + wt * d * norms + gate
    if case["train"]:
        b += T * d * (r + (2 + r if case["pre"] else 0) + 2 + r + 2) + wt * d * norms + 2 * gate
    return dict(bytes=b, flops=T * d * (4 + 4 * norms + (8 + 12 * norms if case["train"] else 0)))


# ------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] in ("route", "replay"):
        return _exact_route(case, st)
    return _exact_norm(case, st) if case["kind"] == "norm" else _exact_join(case, st)


def _exact_route(case, st):
    T, E, k = case["T"], case["E"], case["k"]
    l, D = st["logits"].double(), torch.float64
    off = st["logits"] <= torch.finfo(st["logits"].dtype).min
    if case["score"] == "sigmoid":
        s = torch.sigmoid(l)
    else:
        s = torch.softmax(l.masked_fill(off, -math.inf), dim=1)
        s = s.masked_fill(off.all(dim=1, keepdim=True), 0.0)
    s = s.masked_fill(off, 0.0)
    r = {}
    if case["kind"] == "replay":
        ids = st["rec"][1, :, st["s0"]:st["s0"] + T].t().long()
    else:
        c = s.float()
        if st["bias"] is not None:
            c = c + st["bias"]
        c = c.masked_fill(off, -math.inf)
        G, S = case["groups"], E // case["groups"]
        left = torch.ones((T, E), dtype=torch.bool, device=DEV)
        if G > 1:
            parts = c.reshape(T, G, S)
            first, at = parts.max(dim=2)
            value = first
            if case["group_top"] == 2:
                again = parts.scatter(2, at.unsqueeze(2), -math.inf).amax(dim=2)
                value = torch.where(again > -math.inf, first + again, first)
            ahead = torch.zeros((T, G), dtype=torch.int32, device=DEV)   # how many groups come before each
            for g in range(G):
                v = value[:, g:g + 1]
                tie = torch.arange(G, device=DEV) > g
                ahead += ((v > value) | ((v == value) & tie)).int()
            left = (ahead < case["top_groups"]).unsqueeze(2).expand(T, G, S).reshape(T, E).clone()
        number = torch.arange(E, device=DEV).expand(T, E)
        picks = []
        for _ in range(k):
            best = c.masked_fill(~left, -math.inf).amax(dim=1, keepdim=True)
            pick = torch.where(left & (c == best), number, E).amin(dim=1, keepdim=True)
            left.scatter_(1, pick, False)
            picks.append(pick)
        ids = torch.cat(picks, dim=1)
        if case["capture"]:
            r["rec"] = st["rec"].clone()
            for j in range(k):
                r["rec"][2, j, 50:50 + T] = ids[:, j].int()
        if case["balance"]:
            load = torch.bincount(ids.reshape(-1), minlength=E).to(D)
            r["bias"] = st["bias"].to(D) + STEP * torch.sign(load.mean() - load)
    pick = torch.gather(s, 1, ids)
    div = pick.sum(dim=1, keepdim=True) if case["renorm"] else torch.ones((T, 1), dtype=D, device=DEV)
    div = torch.where(div > 0, div, torch.full_like(div, math.inf))
    w = case["scale"] * pick / div
    r["ids"], r["w"] = ids.int(), w
    if case["train"]:
        # through the weights to the scores, then through the scores
        dw = st["d_w"].to(D)
        ds = case["scale"] * dw
        if case["renorm"]:
            ds = (ds - (dw * w).sum(dim=1, keepdim=True)) / div
        full = torch.zeros((T, E), dtype=D, device=DEV)
        for j in range(k):
            full.scatter_add_(1, ids[:, j:j + 1], ds[:, j:j + 1])
        if case["score"] == "sigmoid":
            r["d_logits"] = full * s * torch.sigmoid(-l)
        else:
            r["d_logits"] = s * (full - (s * full).sum(dim=1, keepdim=True))
    return r


def _unit(v):
    """(v over its root mean square, that) of rows in 64 bits."""
    rms = (v.square().sum(dim=1, keepdim=True) / v.shape[1] + EPS).sqrt()
    return v / rms, rms


def _through(da, u, rms):
    return (da - u * ((da * u).sum(dim=1, keepdim=True) / u.shape[1])) / rms


def _exact_norm(case, st):
    u, rms = _unit(st["x"].double())
    w = st["w"].double()
    r = dict(h=u * w)
    if case["train"]:
        dh = st["dh"].double()
        r["dx"] = _through(dh * w, u, rms) + (0.0 if st["add"] is None else st["add"].double())
        r["dw"] = (dh * u).sum(dim=0)
    return r


def _exact_join(case, st):
    y, r0 = st["y"].double(), st["r"].double()
    T, d = y.shape
    u, rms = _unit(y) if case["post"] else (y, None)
    wp = st["w_post"].double() if case["post"] else torch.ones(d, dtype=torch.float64, device=DEV)
    raw = st["gate"]
    if raw is None:
        g = slope = torch.ones((1, 1), dtype=torch.float64, device=DEV)
    else:
        g = raw.double().reshape(dict(channel=(1, d), token=(T, 1), full=(T, d))[case["gate"]])
        slope = torch.ones_like(g)
        if case["act"] == "sigmoid":
            slope = torch.sigmoid(g) * torch.sigmoid(-g)
            g = torch.sigmoid(g)
    r1 = r0 * case["r_scale"] + u * wp * g * case["y_scale"]
    out = dict(r=r1)
    kept = r1.to(st["r"].dtype).double()   # the stream goes on as it is stored
    if case["pre"]:
        v, rms1 = _unit(kept)
        out["h"] = v * st["w_pre"].double()
    if not case["train"]:
        return out
    D = st["d_out"].double()
    if case["pre"]:
        dh = st["dh"].double()
        D = D + _through(dh * st["w_pre"].double(), v, rms1)
        out["dw_pre"] = (dh * v).sum(dim=0)
    out["dr"] = D * case["r_scale"]
    D = D * case["y_scale"]
    if raw is not None:
        dg = D * u * wp * slope
        out["dgate"] = dict(channel=lambda: dg.sum(dim=0), token=lambda: dg.sum(dim=1), full=lambda: dg)[case["gate"]]()
    D = D * g
    if case["post"]:
        out["dw_post"] = (D * u).sum(dim=0)
        D = _through(D * wp, u, rms)
    out["dy"] = D
    return out
