"""CPU checks of the norms' C entry points: refusals before any launch, no-ops,
workspace sizes."""

import ctypes
import os

import pytest

from moe_expert_layer_r3_amd import ops

pytestmark = pytest.mark.skipif(not os.path.exists(ops.LIB_PATH), reason="library not built")

P = ctypes.c_void_p
A = P(0x1000)      # 16-byte aligned, never dereferenced
ODD = P(0x1008)    # 8-byte aligned only
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def rc(name, args, **kw):
    a = dict(args)
    for k in kw:
        assert k in a, k
    a.update(kw)
    return getattr(ops.lib(), name)(*a.values())


NORM = dict(x=A, xt=0, ldx=64, w=A, wt=0, T=4, d=64, eps=1e-6, h=A, rstd=None, s=None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), -2), (dict(T=(1 << 30) + 1), -2), (dict(d=0), -2), (dict(d=60), -2), (dict(d=(1 << 20) + 8), -2),
    (dict(xt=2), -3), (dict(wt=-1), -3), (dict(eps=0.0), -2), (dict(eps=-1.0), -2), (dict(eps=NAN), -2), (dict(eps=INF), -2),
    (dict(x=None), -1), (dict(w=None), -1), (dict(h=None), -1), (dict(ldx=56), -2), (dict(ldx=68), -2),
    (dict(ldx=(1 << 22) + 8), -2), (dict(x=ODD), -2), (dict(w=ODD), -2), (dict(h=ODD), -2), (dict(T=0, x=None, h=None), 0),
])
def test_norm_refusals(kw, want):
    assert rc("moe_norm", NORM, **kw) == want
    assert want == 0 or ops.last_error()


NORMB = dict(dh=A, x=A, xt=0, ldx=64, w=A, wt=0, rstd=A, add=None, T=4, d=64, dx=A, dw=A, ws=A, wsb=BIG, s=None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), -2), (dict(d=12), -2), (dict(xt=3), -3), (dict(wt=3), -3), (dict(dh=None), -1), (dict(x=None), -1),
    (dict(w=None), -1), (dict(rstd=None), -1), (dict(ldx=68), -2), (dict(ldx=32), -2), (dict(dh=ODD), -2), (dict(x=ODD), -2),
    (dict(add=ODD), -2), (dict(dx=ODD), -2), (dict(dw=ODD), -2), (dict(ws=ODD), -2), (dict(ws=None), -1), (dict(wsb=16), -4),
    (dict(dx=None, dw=None), 0), (dict(T=0, dh=None, x=None, dw=None), 0),
])
def test_norm_backward_refusals(kw, want):
    assert rc("moe_norm_backward", NORMB, **kw) == want


JOIN = dict(y=A, ldy=64, r=A, rt=0, ldr=64, wp=A, g=A, gk=1, gt=0, ga=0, rs=1.0, ys=1.0, wn=A, wt=0, T=4, d=64, eps=1e-6,
            out=A, h=A, sp=None, sn=None, s=None)
B = P(0x100000)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), -2), (dict(d=4), -2), (dict(rt=2), -3), (dict(wt=2), -3), (dict(gk=4), -3), (dict(gk=-1), -3),
    (dict(gt=2), -3), (dict(ga=1), -3), (dict(ga=2), -3), (dict(g=None), -1), (dict(g=ODD), -2), (dict(eps=0.0), -2),
    (dict(rs=NAN), -2), (dict(ys=INF), -2), (dict(y=None), -1), (dict(r=None), -1), (dict(out=None), -1), (dict(h=None), -1),
    (dict(ldy=60), -2), (dict(ldr=32), -2), (dict(ldr=72), -2), (dict(y=ODD), -2), (dict(r=ODD), -2), (dict(out=ODD), -2),
    (dict(wp=ODD), -2), (dict(wn=ODD), -2), (dict(h=ODD), -2), (dict(T=0, y=None, r=None, out=None, h=None, g=None), 0),
])
def test_join_refusals(kw, want):
    assert rc("moe_join", JOIN, **kw) == want


JOINB = dict(do=A, dh=A, y=A, ldy=64, r=A, rt=0, wp=A, g=A, gk=1, gt=0, ga=0, rs=1.0, ys=1.0, wn=A, wt=0, sp=A, sn=A, T=4,
             d=64, dr=A, dy=A, dwp=A, dwn=A, dg=A, ws=A, wsb=BIG, s=None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), -2), (dict(d=4), -2), (dict(rt=2), -3), (dict(wt=2), -3), (dict(gk=4), -3), (dict(gt=2), -3),
    (dict(ga=3), -3), (dict(g=None), -1), (dict(g=ODD), -2), (dict(rs=NAN), -2), (dict(y=None), -1), (dict(dh=None), -1),
    (dict(wn=None), -1), (dict(do=None, dh=None, wn=None, dwn=None), -1), (dict(r=None), -1), (dict(sn=None), -1),
    (dict(sp=None), -1), (dict(wp=None), -1), (dict(gk=0), -1), (dict(ldy=60), -2), (dict(do=ODD), -2), (dict(dh=ODD), -2),
    (dict(y=ODD), -2), (dict(r=ODD), -2), (dict(dr=ODD), -2), (dict(dy=ODD), -2), (dict(dwp=ODD), -2), (dict(dwn=ODD), -2),
    (dict(dg=ODD), -2), (dict(ws=ODD), -2), (dict(ws=None), -1), (dict(wsb=64), -4),
    (dict(dr=None, dy=None, dwp=None, dwn=None, dg=None), 0),
    (dict(T=0, do=None, dh=None, y=None, r=None, g=None, dwp=None, dwn=None, dg=None), 0),
])
def test_join_backward_refusals(kw, want):
    assert rc("moe_join_backward", JOINB, **kw) == want


def test_workspaces():
    """No rows, no workspace; it grows with the rows up to a bound, and with what is summed."""
    one = lambda T, d: ops.workspace_bytes("moe_norm_backward_workspace", T, d)
    assert one(0, 64) == 0 and one(1, 64) > 0
    assert one(1 << 30, 64) == one(1 << 20, 64)
    assert one(1 << 30, 1 << 20) <= 1 << 30
    assert ops.workspace_bytes("moe_join_backward_workspace", 100, 64) >= one(100, 64)
    for bad in ((-1, 64), (4, 60), (4, (1 << 20) + 8)):
        with pytest.raises(ops.MoeError):
            one(*bad)
