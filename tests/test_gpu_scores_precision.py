"""The 64 bits of scored routing's weights and gradients on the GPU, where fewer would
show: bounds of their own, next to those of scores_ref.

u = 2^-24. What is rounded once from 64 bits is off by u of itself (2^-8 in bf16,
and u for the way through fp32), or half the smallest step. In front of that
rounding stand some 20 operations of 2^-53 each, an exponential good to 2^-49 and a
reciprocal good to 2^-50: 2^-46 of the terms that a difference is taken of."""

import numpy as np
import pytest
import torch

import scores_ref as R
from gpu_util import DEV, np64, say
from moe_expert_layer_r3_amd import ops
from test_gpu_scores import close

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balanced_gradients(score):
    """d_w of the last pick next to the mean of all, so that its gradient is some 2^-24
    of the terms it is a difference of."""
    T, E, k = 8192, 32, 3
    say(f"balanced gradients {score}")
    rng = np.random.default_rng(41)
    lg = torch.tensor(rng.standard_normal((T, E)) * 1.5).float().to(DEV)
    ids = np.ascontiguousarray(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32))
    l = np64(lg)
    s = R.scores(l, "f32", score)
    _, share = R.weights(l, s, "f32", ids, score, True, 1.0)
    d_w = rng.standard_normal((T, k)).astype(np.float32)
    d_w[:, 2] = (share[:, :2] * d_w[:, :2]).sum(axis=1) / share[:, :2].sum(axis=1)
    got = ops.route_scored_backward(torch.tensor(d_w).to(DEV), lg, torch.tensor(ids).to(DEV), ops.Scoring(score))
    g, size = R.gradient(l, s, "f32", ids, d_w.astype(np.float64), score, True, 1.0)
    close(got, g, R.ROUND["f32"] * np.abs(g) + R.TINY["f32"] + 2.0 ** -46 * size, "d_logits")


def test_sigmoid_scores_at_the_end_of_64_bits():
    """Logits from -706 to the border below which scores are 0: weights of equal ones are 1 / k,
    those of others their exponentials' shares."""
    border = 709.782712893384
    l = -np.concatenate([np.arange(706.0, 712.0, 0.01), [708.39, 708.4, 709.0, 709.01, 709.78, 709.79]]).astype(np.float32)
    T, E, k = len(l), 8, 4
    lg = np.repeat(l[:, None], E, axis=1)
    lg[:, 1] = lg[:, 0] + np.float32(1.0)
    x = lg.astype(np.float64)
    ids = np.tile(np.arange(k, dtype=np.int32), (T, 1))
    there = x[:, :k] >= -border
    e = np.where(there, np.exp(x[:, :k] - x[:, 1:2]), 0.0)       # sigmoid(l) = exp(l) (1 - 2^-1000)
    total = e.sum(axis=1, keepdims=True)
    want = np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))
    rec = torch.tensor(np.ascontiguousarray(ids.T[None])).to(DEV)
    _, w = ops.replay_scored(rec, 0, 0, torch.tensor(lg).to(DEV), ops.Scoring("sigmoid"))
    # scores down to 2^-1024 are subnormal: off by half a step of 2^-1074, 2^-51 of them and less
    close(w, want, (R.ROUND["f32"] + 2.0 ** -46) * want, "w")


def softmax_rows(T, E, seed):
    """Rows of which a third are normal, a third have one logit in front and all others equal
    (their exponentials' errors have one sign), a third one logit far in front."""
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((T, E)) * 1.5
    flat = l[1::3]
    flat[:] = rng.uniform(-6.0, 0.0, size=(len(flat), 1))
    flat[np.arange(len(flat)), rng.integers(0, E, size=len(flat))] = 0.3
    far = l[2::3]
    far[np.arange(len(far)), rng.integers(0, E, size=len(far))] += rng.uniform(8.0, 25.0, size=len(far))
    return l


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,groups,top_groups", [
    (1200, 3, 2, 1, 1), (1200, 16, 2, 1, 1), (9000, 60, 6, 5, 2), (1200, 128, 8, 1, 1), (9000, 256, 8, 8, 4), (9000, 256, 8, 1, 1),
    (600, 256, 16, 1, 1), (1200, 256, 16, 16, 5), (1200, 512, 8, 16, 4), (9000, 510, 8, 1, 1), (600, 1024, 16, 1, 1),
    (600, 1000, 8, 40, 11), (1, 256, 8, 8, 4)])
def test_softmax_weights_are_rounded_once(kind, T, E, k, groups, top_groups):
    """Weights that are not renormalised: scores of the whole row, rounded once from 64 bits."""
    say(f"softmax weights T={T} E={E} k={k} {kind}")
    lg = torch.tensor(softmax_rows(T, E, 42)).to(dict(f32=torch.float32, bf16=torch.bfloat16)[kind]).to(DEV)
    l = np64(lg)
    s = R.scores(l, kind, "softmax")
    rec = torch.zeros((1, k, T), dtype=torch.int32, device=DEV)
    for bias in (None, torch.tensor(np.random.default_rng(43).standard_normal(E).astype(np.float32) * 0.05).to(DEV)):
        sc = ops.Scoring("softmax", groups=groups, top_groups=top_groups, renorm=False, scale=1.5)
        ids, w = ops.route_scored(lg, k, sc, bias=bias, capture=(rec, 0, 0))
        want, _ = R.weights(l, s, kind, ids.cpu().numpy(), "softmax", False, 1.5)
        tol = (R.ROUND["f32"] + 2.0 ** -46) * want + R.TINY["f32"]
        close(w, want, tol, "w")
        close(ops.replay_scored(rec, 0, 0, lg, sc)[1], want, tol, "replayed w")


def plain_softmax_gradient(s, ids, d_w, scale):
    """(d_logits, size of the terms of its bracket times the score) of s_e (scale sum d_w - scale dot)."""
    T, E = s.shape
    i64 = ids.astype(np.int64)
    sel = np.take_along_axis(s, i64, axis=1)
    own, big = np.zeros((T, E)), np.zeros((T, E))
    at = (np.repeat(np.arange(T), ids.shape[1]), i64.ravel())
    np.add.at(own, at, scale * d_w.ravel())
    np.add.at(big, at, scale * np.abs(d_w).ravel())
    return (s * (own - scale * (sel * d_w).sum(axis=1, keepdims=True)),
            s * (big + scale * np.abs(sel * d_w).sum(axis=1, keepdims=True)))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(2001, 4, 1), (1203, 60, 2), (1202, 64, 1), (3001, 256, 1), (3001, 256, 8), (801, 510, 3),
                                   (803, 1024, 1), (803, 1000, 16), (1, 256, 1)])
def test_plain_softmax_gradients_of_confident_rows(kind, T, E, k):
    """Gaps up to 25 between the largest logit and the rest: its gradient is scale d_w s (1 - s).
    Five roundings to 32 bits (bracket, 1 / sum, exponential, two products), then that to bf16."""
    scale = 1.5
    for chosen in ("best", "any", "twice"):
        say(f"plain softmax gradient T={T} E={E} k={k} {kind} {chosen}")
        rng = np.random.default_rng(44)
        lg = torch.tensor(softmax_rows(T, E, 45)).to(dict(f32=torch.float32, bf16=torch.bfloat16)[kind]).to(DEV)
        l = np64(lg)
        s = R.scores(l, kind, "softmax")
        order = np.argsort(-l if chosen == "best" else rng.random((T, E)), axis=1, kind="stable")
        ids = np.ascontiguousarray(order[:, :k].astype(np.int32))
        if chosen == "twice":
            ids[:, k // 2:] = order[:, :1]
        d_w = (0.5 + rng.random((T, k))).astype(np.float32)
        d_w[::2] = d_w[::2, :1]
        got = ops.route_scored_backward(torch.tensor(d_w).to(DEV), lg, torch.tensor(ids).to(DEV),
                                        ops.Scoring("softmax", renorm=False, scale=scale))
        g, size = plain_softmax_gradient(s, ids, d_w.astype(np.float64), scale)
        tol = (5 * U * 1.001 + (R.ROUND["bf16"] if kind == "bf16" else 0.0)) * np.abs(g) + R.TINY[kind] + 2.0 ** -46 * size
        close(got, g, tol, "d_logits")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("E,k", [(9, 3), (64, 4), (256, 8), (510, 2), (1000, 16)])
def test_gradients_of_odd_logits(score, renorm, E, k, kind):
    """NaN and infinite logits, masked experts among the chosen ones, ids outside [0, E): NaN
    where a score is NaN in the formula, 0 at masked experts and for tokens with such an id."""
    say(f"odd gradients {score} renorm={renorm} E={E} k={k} {kind}")
    T, scale = 403, 1.5
    rng = np.random.default_rng(46)
    l = rng.standard_normal((T, E)) * 1.3
    l[rng.random((T, E)) < 0.2] = -np.inf
    l[rng.random((T, E)) < 0.1] = R.LOWEST[kind]
    odd = rng.random((T, E)) < 0.5 / E
    l[odd] = rng.choice([np.nan, np.inf], size=odd.sum())
    l[5] = np.nan
    l[6] = -np.inf
    l[7], l[7, 1::2] = -np.inf, np.inf
    l[8], l[8, ::3] = np.nan, R.LOWEST[kind]
    lg = torch.tensor(l).to(dict(f32=torch.float32, bf16=torch.bfloat16)[kind]).to(DEV)
    ids = np.ascontiguousarray(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32))
    ids[3::11, k // 2] = rng.choice([-1, E, E + 5, -(1 << 31), (1 << 31) - 1], size=len(ids[3::11]))
    bad = ((ids < 0) | (ids >= E)).any(axis=1)
    assert bad[(np.isnan(l) | (l == np.inf)).any(axis=1)].any()
    d_w = rng.standard_normal((T, k)).astype(np.float32)
    got = ops.route_scored_backward(torch.tensor(d_w).to(DEV), lg, torch.tensor(ids).to(DEV),
                                    ops.Scoring(score, renorm=renorm, scale=scale))
    l, dw = np64(lg), d_w.astype(np.float64)
    i64 = np.where(bad[:, None], 0, ids).astype(np.int64)
    with np.errstate(invalid="ignore", over="ignore"):
        s = R.scores(l, kind, score)
        if score == "softmax":
            s = np.where((l == np.inf).any(axis=1, keepdims=True) & ~R.masked(l, kind), np.nan, s)
        if score == "softmax" and not renorm:
            g, size = plain_softmax_gradient(s, i64, dw, scale)
        else:
            if score == "softmax" and renorm:      # of the chosen logits alone
                some = np.isnan(np.take_along_axis(l, i64, axis=1)) | (np.take_along_axis(l, i64, axis=1) == np.inf)
                _, share = R.weights(l, s, kind, i64, score, True, scale)
                share = np.where(some.any(axis=1, keepdims=True), np.nan, share)
            else:
                _, share = R.weights(l, s, kind, i64, score, renorm, scale)
            dot = (share * dw).sum(axis=1, keepdims=True) if renorm else 0.0
            own = scale * share * (dw - dot)
            size = np.abs(scale * share * dw)
            if renorm:
                size = size + np.abs(scale * share) * np.abs(share * dw).sum(axis=1, keepdims=True)
            if score == "sigmoid":
                far = 1.0 / (1.0 + np.exp(np.take_along_axis(l, i64, axis=1)))
                own, size = own * far, size * far
            g, big = np.zeros((T, E)), np.zeros((T, E))
            np.put_along_axis(g, i64, own, axis=1)
            np.put_along_axis(big, i64, size, axis=1)
            size = big
    g, size = np.where(R.masked(l, kind), 0.0, g), np.where(R.masked(l, kind), 0.0, size)
    g[bad], size[bad] = 0.0, 0.0
    tol = (5 * U * 1.001 + R.ROUND[kind]) * np.abs(g) + R.TINY[kind] + 2.0 ** -46 * size
    close(got, g, tol, "d_logits")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("E,k", [(16, 4), (256, 8), (600, 3)])
def test_weights_of_very_negative_logits(score, renorm, E, k, kind):
    """Scores next to fp32's smallest values and below them: chosen where nothing larger is there
    (sigmoid), and replayed, of softmax next to a large one."""
    say(f"very negative {score} renorm={renorm} E={E} k={k} {kind}")
    T = 300
    rng = np.random.default_rng(47)
    l = rng.uniform(-106.0, -84.0, size=(T, E))
    if score == "softmax":
        l[:, 0] = 0.0
    lg = torch.tensor(l).to(dict(f32=torch.float32, bf16=torch.bfloat16)[kind]).to(DEV)
    l = np64(lg)
    s = R.scores(l, kind, score)
    sc = ops.Scoring(score, renorm=renorm)
    if score == "sigmoid":
        ids, w = ops.route_scored(lg, k, sc)
        ref = R.choices(l, s, kind, k)
        assert np.array_equal(ids.cpu().numpy(), ref)
        want, _ = R.weights(l, s, kind, ref, score, renorm, 1.0)
        close(w, want, (R.ROUND["f32"] + 2.0 ** -46) * want + R.TINY["f32"], "w")
    ids = np.ascontiguousarray(1 + np.argsort(rng.random((T, E - 1)), axis=1)[:, :k].astype(np.int32))
    rec = torch.tensor(np.ascontiguousarray(ids.T[None])).to(DEV)
    _, w = ops.replay_scored(rec, 0, 0, lg, sc)
    want, _ = R.weights(l, s, kind, ids, score, renorm, 1.0)
    assert renorm or want.min() < 2.0 ** -145 < 2.0 ** -126 < want.max()    # subnormal ones and others
    close(w, want, (R.ROUND["f32"] + 2.0 ** -46) * want + R.TINY["f32"], "replayed w")
