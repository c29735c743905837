"""CPU checks of the scored routing's C entry points and Python forms: refusals
before any launch, and no-ops."""

import ctypes
import os

import pytest
import torch

from moe_expert_layer_r3_amd import ops

pytestmark = pytest.mark.skipif(not os.path.exists(ops.LIB_PATH), reason="library not built")

P = ctypes.c_void_p
A = P(0x1000)      # 16-byte aligned, never dereferenced
ODD = P(0x1008)    # 8-byte aligned only


def rc(name, args, **kw):
    a = dict(args)
    for k in kw:
        assert k in a, k
    a.update(kw)
    return getattr(ops.lib(), name)(*a.values())


ROUTE = dict(l=A, lt=1, T=4, E=16, k=2, score=1, bias=None, groups=4, top=2, gtop=2, renorm=1, scale=1.0, ids=A, w=A,
             load=None, rec=None, NL=0, S=0, layer=0, s0=0, s=None)
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), -2), (dict(T=(1 << 30) + 1), -2), (dict(E=0), -2), (dict(E=1025, groups=1, top=1), -2), (dict(k=0), -2),
    (dict(k=17), -2), (dict(E=8, k=9), -2), (dict(lt=2), -3), (dict(score=2), -3), (dict(score=-1), -3),
    (dict(groups=0), -2), (dict(groups=3), -2), (dict(groups=65), -2), (dict(E=130, groups=65), -2), (dict(top=0), -2),
    (dict(top=5), -2), (dict(k=9), -2), (dict(gtop=0), -2), (dict(gtop=3), -2), (dict(scale=NAN), -2), (dict(scale=INF), -2),
    (dict(l=None), -1), (dict(ids=None), -1), (dict(w=None), -1), (dict(l=ODD), -2),
    (dict(rec=A, NL=4, S=100, layer=4), -2), (dict(rec=A, NL=4, S=100, layer=-1), -2), (dict(rec=A, NL=0, S=100), -2),
    (dict(rec=A, NL=4, S=100, s0=97), -2), (dict(rec=A, NL=4, S=100, s0=-1), -2), (dict(rec=A, NL=4, S=3), -2),
    (dict(rec=A, NL=4, S=1 << 62, s0=(1 << 63) - 1), -2),
    (dict(T=0, l=None, ids=None, w=None), 0),
])
def test_route_refusals(kw, want):
    assert rc("moe_route_scored", ROUTE, **kw) == want
    assert want == 0 or ops.last_error()


REPLAY = dict(rec=A, NL=4, k=2, S=100, layer=0, s0=0, T=4, l=A, lt=1, E=16, score=1, renorm=1, scale=1.0, ids=A, w=A,
              st=None, s=None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), -2), (dict(k=17), -2), (dict(k=0), -2), (dict(E=0), -2), (dict(E=1), -2), (dict(layer=4), -2),
    (dict(layer=-1), -2), (dict(NL=0), -2), (dict(s0=97), -2), (dict(s0=-1), -2), (dict(S=3), -2), (dict(lt=5), -3),
    (dict(score=3), -3), (dict(scale=INF), -2), (dict(rec=None), -1), (dict(l=None), -1), (dict(ids=None), -1),
    (dict(w=None), -1), (dict(l=ODD), -2), (dict(s0=(1 << 63) - 1), -2), (dict(T=0, rec=None, l=None), 0),
])
def test_replay_refusals(kw, want):
    assert rc("moe_replay_scored", REPLAY, **kw) == want


BACK = dict(dw=A, l=A, lt=1, ids=A, T=4, k=2, E=16, score=1, renorm=1, scale=1.0, out=A, s=None)
PARTS = dict(part=A, pr=A, cap=128, d=256, l=A, lt=1, ids=A, T=4, k=2, E=16, score=1, renorm=1, scale=1.0, dg=A, out=A,
             s=None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), -2), (dict(k=0), -2), (dict(E=1025), -2), (dict(lt=2), -3), (dict(score=2), -3), (dict(scale=NAN), -2),
    (dict(l=None), -1), (dict(ids=None), -1), (dict(out=None), -1), (dict(l=ODD), -2), (dict(out=ODD), -2),
    (dict(T=0, l=None, ids=None, out=None), 0),
])
def test_backward_refusals(kw, want):
    assert rc("moe_route_scored_backward", BACK, **kw) == want
    assert rc("moe_route_scored_backward_parts", PARTS, **kw) == want


def test_more_backward_refusals():
    assert rc("moe_route_scored_backward", BACK, dw=None) == -1
    for kw, want in ((dict(part=None), -1), (dict(pr=None), -1), (dict(dg=None), -1), (dict(d=100), -2), (dict(d=0), -2),
                     (dict(cap=-1), -2)):
        assert rc("moe_route_scored_backward_parts", PARTS, **kw) == want


def test_balance_refusals():
    base = dict(load=A, bias=A, E=16, step=0.1, clear=1, out=A, s=None)
    for kw, want in ((dict(E=0), -2), (dict(E=1025), -2), (dict(step=NAN), -2), (dict(load=None), -1), (dict(bias=None), -1),
                     (dict(out=None), -1)):
        assert rc("moe_balance_bias", base, **kw) == want


def test_python_refusals():
    with pytest.raises(ValueError):
        ops.Scoring("tanh")
    lg = torch.zeros(4, 16)
    with pytest.raises(ValueError):
        ops.route_scored(lg, 2, ops.Scoring())       # not on the GPU
    with pytest.raises(TypeError):
        ops.route_scored(lg.double(), 2, ops.Scoring())
    with pytest.raises(ValueError):
        ops.record_args(torch.zeros(2, 3, 4, dtype=torch.int32), 0, 0, 2, torch.device("cpu"))
    with pytest.raises(ValueError):
        ops.record_args(torch.zeros(2, 2, 4, dtype=torch.int64), 0, 0, 2, torch.device("cpu"))


def test_the_references_agree():
    """The reference for many tokens at once against the one that goes token by token."""
    import numpy as np

    import scores_ref as R
    rng = np.random.default_rng(5)
    for E, k, groups, top, gt in ((16, 4, 4, 2, 2), (24, 6, 3, 2, 1), (9, 9, 1, 1, 2), (32, 3, 16, 3, 2)):
        l = np.round(rng.standard_normal((60, E)) * 2) / 2
        l[rng.random((60, E)) < 0.3] = -np.inf
        l[rng.random((60, E)) < 0.1] = R.LOWEST["f32"]
        l[rng.random((60, E)) < 0.05] = np.nan
        l[::7] = -np.inf
        for score in ("sigmoid", "softmax"):
            s = R.scores(l, "f32", score)
            for bias in (None, np.round(rng.standard_normal(E), 1)):
                a = (l, s, "f32", k, bias, groups, top, gt)
                assert np.array_equal(R.choice(*a), R.choices(*a))
