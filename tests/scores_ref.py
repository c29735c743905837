"""Plain 64-bit forms of routing by scores (not collected by pytest).

Bounds: weights and gradients are computed in 64 bits from a token's own
logits and rounded once, so a value v is off by at most 2^-24 |v| in fp32
(2^-8 |v| in bf16, 2^-24 more for the way through fp32), by half the smallest
step where it is subnormal (steps of 2^-149 in fp32, of 2^-126 / 2^7 = 2^-133 in
bf16: 2^-134, and 2^-150 more for the way through fp32), and by 2^-46 of the terms
it is a difference of (some 20 roundings of 2^-53 and exp's few ulps).

Softmax scores that are not renormalised divide by a sum over the whole row, whose
terms exp(x), x = l - m <= 0, are 32-bit ones: the difference x, its product with
log2 e and the hardware's exp2 (good to one ulp, 2 u with u = 2^-24) make a term off
by at most (2 |x| + 3) u of itself; the sum (in 64 bits) is then off by the mean of
that weighted with exp(x) / sum, and the mean |x| is ln E at most (it is the
distribution's entropy less ln sum): (2 ln E + 3) u (row_err). A gradient's own score
is such a term over such a sum: (2 |x| + 2 ln E + 6) u."""

import numpy as np

LOWEST = {"f32": -3.4028234663852886e38, "bf16": -3.3895313892515355e38}
ROUND = {"f32": 2.0 ** -24 * 1.001, "bf16": (2.0 ** -8 + 2.0 ** -24) * 1.001}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -134 + 2.0 ** -150}
U = 2.0 ** -24


def row_err(E, score, renorm):
    return (2 * np.log(E) + 3) * U if score == "softmax" and not renorm else 0.0


def masked(l, kind):
    with np.errstate(invalid="ignore"):
        return l <= LOWEST[kind]


def scores(l, kind, score):
    """fp64 scores [T, E] of logits l (fp64)."""
    off = masked(l, kind)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            v = np.where(off, -np.inf, l)
            m = v.max(axis=1, keepdims=True)
            none = off.all(axis=1, keepdims=True)
            e = np.where(off, 0.0, np.exp(v - np.where(none, 0.0, m)))
            s = e / np.where(none, 1.0, e.sum(axis=1, keepdims=True))
            s = np.where(np.isnan(l).any(axis=1, keepdims=True), np.nan, s)
    return np.where(off, 0.0, s)


def choice(l, s, kind, k, bias=None, groups=1, top_groups=1, group_top=2):
    """ids [T, k] of fp64 scores rounded to fp32."""
    T, E = l.shape
    with np.errstate(invalid="ignore", over="ignore"):
        c = s.astype(np.float32)
        if bias is not None:
            c = c + bias[None, :].astype(np.float32)
        c = np.where(masked(l, kind), np.float32(-np.inf), c)
        S = E // groups
        ids = np.empty((T, k), dtype=np.int32)
        for t in range(T):
            stay = np.ones(groups, dtype=bool)
            if groups > 1:
                value = []
                for g in range(groups):
                    v = c[t, g * S:(g + 1) * S]
                    v = np.sort(v[v > -np.inf])[::-1][:group_top]
                    value.append(np.float32(-np.inf) if v.size == 0 else v[0] if v.size == 1 else np.float32(v[0] + v[1]))
                order = sorted(range(groups), key=lambda g: (-value[g], g))
                stay[:] = False
                stay[order[:top_groups]] = True
            key = lambda e: (bool(np.isnan(c[t, e])), 0.0 if np.isnan(c[t, e]) else -float(c[t, e]), e)
            ids[t] = sorted((e for e in range(E) if stay[e // S]), key=key)[:k]
    return ids


def choices(l, s, kind, k, bias=None, groups=1, top_groups=1, group_top=2):
    """The same for many tokens at once."""
    T, E = l.shape
    with np.errstate(invalid="ignore", over="ignore"):
        c = s.astype(np.float32)
        if bias is not None:
            c = c + bias[None, :].astype(np.float32)
        c = np.where(masked(l, kind), np.float32(-np.inf), c)
        out = np.zeros((T, E), dtype=bool)
        if groups > 1 and top_groups < groups:
            v = np.where(np.isnan(c), np.float32(-np.inf), c).reshape(T, groups, E // groups)
            v = -np.sort(-v, axis=2)[:, :, :group_top]
            value = np.where(v > -np.inf, v, np.float32(0)).sum(axis=2, dtype=np.float32)
            value[v[:, :, 0] == -np.inf] = -np.inf
            place = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1, kind="stable")
            out = np.repeat(place >= top_groups, E // groups, axis=1)
        last = np.isnan(c)
        key = np.where(last, 0.0, -c.astype(np.float64))
        e = np.broadcast_to(np.arange(E), (T, E))
        return np.lexsort((e, key, last, out), axis=1)[:, :k].astype(np.int32)


def weights(l, s, kind, ids, score, renorm, scale):
    """fp64 (weights, shares) [T, k]."""
    sel = np.take_along_axis(s, ids.astype(np.int64), axis=1)
    if not renorm:
        return scale * sel, sel
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if score == "softmax":
            v = np.take_along_axis(np.where(masked(l, kind), -np.inf, l), ids.astype(np.int64), axis=1)
            m = v.max(axis=1, keepdims=True)
            sel = np.where(v == -np.inf, 0.0, np.exp(v - np.where(m == -np.inf, 0.0, m)))
        total = sel.sum(axis=1, keepdims=True)
        share = np.where(total == 0, 0.0, sel / total)
    return scale * share, share


def gradient(l, s, kind, ids, d_w, score, renorm, scale):
    """(d_logits [T, E], size of the terms each is a difference of) in fp64."""
    T, E = l.shape
    _, share = weights(l, s, kind, ids, score, renorm, scale)
    i64 = ids.astype(np.int64)
    dot = (share * d_w).sum(axis=1, keepdims=True)
    size = scale * share * (np.abs(d_w) + (np.abs(share * d_w).sum(axis=1, keepdims=True)))
    g = scale * share * (d_w - (dot if renorm else 0.0))
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            far = 1.0 / (1.0 + np.exp(np.take_along_axis(l, i64, axis=1)))
        g, size = g * far, size * far
    out, big = np.zeros((T, E)), np.zeros((T, E))
    rows = np.repeat(np.arange(T), ids.shape[1])
    np.add.at(out, (rows, i64.ravel()), g.ravel())
    np.add.at(big, (rows, i64.ravel()), size.ravel())
    if score == "softmax" and not renorm:
        out -= s * scale * dot
        big += s * scale * np.abs(share * d_w).sum(axis=1, keepdims=True)
        # in units of the 2^-46 that the callers allow: the chosen scores and the row's own
        off = masked(l, kind)
        x = np.where(off, 0.0, l.max(axis=1, keepdims=True) - np.where(off, 0.0, l))
        big *= 1.0 + 2.0 ** 46 * (2 * x + 4 * np.log(E) + 12) * U
    return out, np.abs(big)
