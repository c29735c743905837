"""Cases and plain forms of the layer's dense operators.

Three operators stand around the routed experts of a Mixture-of-Experts layer:
  linear   out = act(x W^T + bias) + residual, and its gradients (the router's
           projection, the second projection of a shared expert)
  ffn      the gated feed-forward block of a shared expert,
           y = (act(x Wg^T + bg) * (x Wu^T + bu)) W2^T + b2 + residual, and its
           gradients from the saved [G, U]
  act8     activations kept in 8 bits between the forward and the backward
           pass: one fp32 scale per row and 128 columns, a = max|v|, s = a / 127,
           q = round(v * (127 / a)), restored as q * s

Weights, biases and their gradients are bf16, as the inputs are; out is bf16 or
fp32.

``own`` chooses between the framework's kernels and elementary torch operations.
"""

import math

import torch

own = False

DEV = "cuda:0"
BF = torch.bfloat16


def listed():
    return [
        # the router of one decoded token: 256 experts' fp32 logits
        dict(name="router_token", kind="linear", T=1, K=7168, N=256, pad=0, act="none", bias=True, residual=False,
             out="f32", train=False),
        # the router over a chunk of prompt tokens
        dict(name="router_prompt", kind="linear", T=8192, K=7168, N=256, pad=0, act="none", bias=True, residual=False,
             out="f32", train=False),
        # an odd projection with everything in the epilogue, reading a column slice of a wider buffer
        dict(name="linear_ragged", kind="linear", T=203, K=520, N=1001, pad=24, act="gelu", bias=True, residual=True,
             out="bf16", train=True),
        # the router in a training step: logits, then gradients from fp32 d_logits
        dict(name="router_train", kind="linear", T=16384, K=7168, N=256, pad=0, act="none", bias=True, residual=False,
             out="f32", train=True),
        # a shared expert on one decoded token, added to the routed experts' sum
        dict(name="ffn_token", kind="ffn", T=1, d=7168, f=2048, act="silu", bias=False, residual=True, save="none"),
        # the same on a decode batch
        dict(name="ffn_batch", kind="ffn", T=48, d=7168, f=2048, act="silu", bias=False, residual=True, save="none"),
        # prompt tokens through a shared expert
        dict(name="ffn_prompt", kind="ffn", T=8192, d=7168, f=2048, act="silu", bias=False, residual=True,
             save="none"),
        # forward and backward of a shared expert at the training step's size
        dict(name="ffn_train", kind="ffn", T=16384, d=7168, f=2048, act="silu", bias=False, residual=True,
             save="bf16"),
        # a small block with odd sizes, biases and another activation
        dict(name="ffn_train_ragged", kind="ffn", T=1237, d=1032, f=344, act="gelu", bias=True, residual=False,
             save="bf16"),
        # the training step with x and [G, U] kept in 8 bits for the backward
        dict(name="ffn_train_act8", kind="ffn", T=16384, d=7168, f=2048, act="silu", bias=False, residual=True,
             save="int8"),
        # one training step's layer input, kept in 8 bits and restored
        dict(name="act8_train", kind="act8", T=16384, d=7168, pad=0),
        # the smallest: 128 rows of 128 columns
        dict(name="act8_small", kind="act8", T=128, d=128, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "ffn", "ffn", "act8"])
    T = _log(rng, 1, 12000)
    act = rng.choice(["none", "relu", "silu", "gelu", "sigmoid"])
    if kind == "linear":
        return dict(kind=kind, T=T, K=8 * _log(rng, 8, 900), N=_log(rng, 1, 6000), pad=8 * rng.choice([0, 0, 1, 5]),
                    act=act, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    out=rng.choice(["bf16", "f32"]), train=rng.random() < 0.5)
    if kind == "ffn":
        save = rng.choice(["none", "bf16", "int8"])
        f = 128 * _log(rng, 1, 16) if save == "int8" else 8 * _log(rng, 8, 256)
        return dict(kind=kind, T=T, d=8 * _log(rng, 8, 900), f=f, act="silu" if act == "none" else act,
                    bias=rng.random() < 0.4, residual=rng.random() < 0.5, save=save)
    return dict(kind=kind, T=T, d=8 * _log(rng, 8, 900), pad=8 * rng.choice([0, 0, 1, 5]))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(shape, std=1.0, dtype=BF):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    T = case["T"]
    st = dict(case=case)
    if case["kind"] == "linear":
        K, N = case["K"], case["N"]
        st["x"] = normal((T, K + case["pad"]))[:, :K]
        st["W"] = normal((N, K), 1.7 / math.sqrt(K))
        st["bias"] = normal((N,), 0.5) if case["bias"] else None
        st["residual"] = normal((T, N)) if case["residual"] else None
        if case["train"]:
            st["dy"] = normal((T, N), 1.0, torch.float32 if case["out"] == "f32" else BF)
        if own:
            from moe_expert_layer_r3_amd.dense import LinearPlan
            st["plan"] = LinearPlan(T, K, N, act=case["act"], out_dtype=torch.float32 if case["out"] == "f32" else BF,
                                    train=case["train"], bias=case["bias"], device=DEV)
    elif case["kind"] == "ffn":
        d, f = case["d"], case["f"]
        st["x"] = normal((T, d))
        st["W13"] = normal((2 * f, d), 1.7 / math.sqrt(d))
        st["W2"] = normal((d, f), 1.0 / math.sqrt(f))
        st["b13"] = normal((2 * f,), 0.5) if case["bias"] else None
        st["b2"] = normal((d,), 0.5) if case["bias"] else None
        st["residual"] = normal((T, d)) if case["residual"] else None
        if case["save"] != "none":
            st["dy"] = normal((T, d))
        if own:
            from moe_expert_layer_r3_amd.dense import GatedFFNPlan
            st["plan"] = GatedFFNPlan(T, d, f, act=case["act"], save=case["save"], bias=case["bias"], device=DEV)
    else:
        # rows of very different size, as residual streams have them
        row = torch.exp(torch.randn((T, 1), generator=g, device=DEV))
        st["x"] = (torch.randn((T, case["d"] + case["pad"]), generator=g, device=DEV) * row).to(BF)[:, :case["d"]]
    return st


def run(state):
    kind = state["case"]["kind"]
    if own:
        return (_own_linear if kind == "linear" else _own_ffn if kind == "ffn" else _own_act8)(state)
    return (_plain_linear if kind == "linear" else _plain_ffn if kind == "ffn" else _plain_act8)(state)


# ------------------------------------------------------------ the framework

def _own_linear(st):
    p = st["plan"]
    out = dict(out=p.forward(st["x"], st["W"], bias=st["bias"], residual=st["residual"]))
    if st["case"]["train"]:
        out["dx"], out["dW"], db = p.backward(st["dy"], st["x"], st["W"])
        if st["bias"] is not None:
            out["db"] = db
    return out


def _own_ffn(st):
    p, save = st["plan"], st["case"]["save"]
    kept = None
    if save == "int8":
        from moe_expert_layer_r3_amd import ops
        kept = ops.act_save(st["x"])
    out = dict(y=p.forward(st["x"], st["W13"], st["W2"], b13=st["b13"], b2=st["b2"], residual=st["residual"]))
    if save == "none":
        return out
    x = st["x"] if kept is None else ops.act_restore(*kept)
    out["dx"], out["dW13"], out["dW2"], db13, db2 = p.backward(st["dy"], x, st["W13"], st["W2"])
    if st["b13"] is not None:
        out["db13"], out["db2"] = db13, db2
    return out


def _own_act8(st):
    from moe_expert_layer_r3_amd import ops
    q, s = ops.act_save(st["x"])
    return dict(restored=ops.act_restore(q, s), scales=s)


# ------------------------------------------------------------ plain forms, in 32 bits

def _act(name, z):
    if name == "relu":
        return torch.clamp_min(z, 0.0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).float()
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if name == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 - s)
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _plain_linear(st):
    c = st["case"]
    x, W = st["x"].float(), st["W"].float()
    z = x @ W.t()
    if st["bias"] is not None:
        z = z + st["bias"].float()
    y = _act(c["act"], z)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    out = dict(out=y if c["out"] == "f32" else y.to(BF))
    if c["train"]:
        # the backward works from the pre-activation kept in bf16
        dz = st["dy"].float()
        if c["act"] != "none":
            dz = dz * _act_slope(c["act"], z.to(BF).float())
        out["dx"] = (dz @ W).to(BF)
        out["dW"] = (dz.t() @ x).to(BF)
        if st["bias"] is not None:
            out["db"] = dz.double().sum(0).to(BF)
    return out


def _plain_keep8(v):
    """(q, s per element) of fp32 rows in blocks of 128 columns, the last one shorter where need be."""
    n, c = v.shape
    nb = (c + 127) // 128
    p = torch.zeros((n, nb * 128), dtype=torch.float32, device=v.device)
    p[:, :c] = v
    p = p.view(n, nb, 128)
    a = torch.clamp_min(p.abs().amax(dim=2, keepdim=True), 2.0 ** -100)
    q = torch.round(p * (127.0 / a))
    s = a / 127.0
    return (q * s).view(n, nb * 128)[:, :c], s.view(n, nb)


def _plain_ffn(st):
    c, f = st["case"], st["case"]["f"]
    x, W13, W2 = st["x"].float(), st["W13"].float(), st["W2"].float()
    gu = x @ W13.t()
    if st["b13"] is not None:
        gu = gu + st["b13"].float()
    h = _act(c["act"], gu[:, :f]) * gu[:, f:]
    y = h @ W2.t()
    if st["b2"] is not None:
        y = y + st["b2"].float()
    if st["residual"] is not None:
        y = y + st["residual"].float()
    out = dict(y=y.to(BF))
    if c["save"] == "none":
        return out
    dy = st["dy"].float()
    if c["save"] == "int8":
        x = _plain_keep8(x)[0].to(BF).float()
        gu = _plain_keep8(gu)[0]
    else:
        gu = gu.to(BF).float()
    G, U = gu[:, :f], gu[:, f:]
    a = _act(c["act"], G)
    dh = dy @ W2
    dgu = torch.cat([dh * U * _act_slope(c["act"], G), dh * a], dim=1)
    out["dx"] = (dgu @ W13).to(BF)
    out["dW13"] = (dgu.t() @ x).to(BF)
    out["dW2"] = (dy.t() @ (a * U)).to(BF)
    if st["b13"] is not None:
        out["db13"] = dgu.double().sum(0).to(BF)
        out["db2"] = dy.double().sum(0).to(BF)
    return out


def _plain_act8(st):
    v, s = _plain_keep8(st["x"].float())
    return dict(restored=v.to(BF), scales=s.t().contiguous())


# ------------------------------------------------------------ what a pass cannot do without

def work(case):
    T = case["T"]
    if case["kind"] == "linear":
        K, N = case["K"], case["N"]
        o = 4 if case["out"] == "f32" else 2
        b = 2 * (T * K + N * K) + o * T * N + (2 * N if case["bias"] else 0) + (2 * T * N if case["residual"] else 0)
        fl = 2 * T * N * K
        if case["train"]:
            b += o * T * N + 2 * (T * K + N * K) + (2 * N if case["bias"] else 0)
            fl *= 3
        return dict(bytes=b, flops=fl)
    d = case["d"]
    if case["kind"] == "ffn":
        f = case["f"]
        b = 2 * (2 * T * d + 3 * f * d) + (2 * (2 * f + d) if case["bias"] else 0) + (2 * T * d if case["residual"] else 0)
        fl = 6 * T * f * d
        if case["save"] != "none":
            b += 2 * (2 * T * d + 3 * f * d) + (2 * (2 * f + d) if case["bias"] else 0)
            fl *= 3
        return dict(bytes=b, flops=fl)
    return dict(bytes=2 * T * d + 2 * T * d + 4 * T * ((d + 127) // 128), flops=4 * T * d)


# ------------------------------------------------------------ the definitions in 64 bits

def _kept(v):
    """What blocks of 128 columns of v stand for in 8 bits, and the blocks' scales."""
    rows, cols = v.shape
    blocks = -(-cols // 128)
    w = torch.nn.functional.pad(v, (0, blocks * 128 - cols)).reshape(rows, blocks, 128)
    top = w.abs().max(dim=2).values.clamp_min(2.0 ** -100)
    # round(v * (127 / a)) as the 32-bit definition has it; values on its border are the same there
    inv = (127.0 / top.float()).double()
    codes = (w.float() * inv.float().unsqueeze(2)).round().double()
    scale = (top.float() / 127.0).double()
    return (codes * scale.unsqueeze(2)).reshape(rows, blocks * 128)[:, :cols], scale


def _value_and_slope(name, z):
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        on = (z > 0).double()
        return z * on, on
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(z * z / -2.0) / math.sqrt(2.0 * math.pi)
    s = torch.sigmoid(z)
    if name == "sigmoid":
        return s, s - s * s
    return z * s, s + z * s * (1.0 - s)


def exact(case, seed):
    st = prepare(case, seed)
    D = lambda n: None if st.get(n) is None else st[n].double()  # noqa: E731
    if case["kind"] == "act8":
        v, s = _kept(D("x"))
        return dict(restored=v, scales=s.t().contiguous())
    x, dy = D("x"), D("dy")
    res = 0.0 if st["residual"] is None else D("residual")
    if case["kind"] == "linear":
        W = D("W")
        z = torch.matmul(x, W.T) + (0.0 if st["bias"] is None else D("bias"))
        r = dict(out=_value_and_slope(case["act"], z)[0] + res)
        if case["train"]:
            dz = dy * _value_and_slope(case["act"], z.to(BF).double())[1]
            r.update(dx=torch.matmul(dz, W), dW=torch.matmul(dz.T, x))
            if st["bias"] is not None:
                r["db"] = dz.sum(dim=0)
        return r
    W13, W2, f = D("W13"), D("W2"), case["f"]
    pre = torch.matmul(x, W13.T) + (0.0 if st["b13"] is None else D("b13"))
    g, u = pre.split(f, dim=1)
    r = dict(y=torch.matmul(_value_and_slope(case["act"], g)[0] * u, W2.T)
             + (0.0 if st["b2"] is None else D("b2")) + res)
    if case["save"] == "none":
        return r
    if case["save"] == "int8":
        pre = torch.cat([_kept(g)[0], _kept(u)[0]], dim=1)
        x = _kept(x)[0].to(BF).double()
    else:
        pre = pre.to(BF).double()
    g, u = pre.split(f, dim=1)
    v, slope = _value_and_slope(case["act"], g)
    dh = torch.matmul(dy, W2)
    dpre = torch.cat([dh * u * slope, dh * v], dim=1)
    r.update(dx=torch.matmul(dpre, W13), dW13=torch.matmul(dpre.T, x), dW2=torch.matmul(dy.T, v * u))
    if st["b13"] is not None:
        r.update(db13=dpre.sum(dim=0), db2=dy.sum(dim=0))
    return r
