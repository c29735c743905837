"""CPU checks of the dense products' C entry points and plans: refusals before
any launch, no-ops, workspace sizes."""

import ctypes
import os

import pytest
import torch

from moe_expert_layer_r3_amd import ops

pytestmark = pytest.mark.skipif(not os.path.exists(ops.LIB_PATH), reason="library not built")

P = ctypes.c_void_p
A = P(0x1000)      # 16-byte aligned, never dereferenced
ODD = P(0x1008)    # 8-byte aligned only
BIG = 1 << 40      # a workspace size that is always enough


def rc(name, args, **kw):
    a = dict(args)
    for k in kw:
        assert k in a, k
    a.update(kw)
    return getattr(ops.lib(), name)(*a.values())


LIN = dict(x=A, ldx=64, W=A, ldw=64, bias=None, res=None, ldr=0, T=4, N=10, K=64, act=0, out=A, ot=0, ldo=10, pre=None,
           ws=A, wsb=BIG, s=None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), -2), (dict(T=(1 << 30) + 1), -2), (dict(N=0), -2), (dict(N=(1 << 20) + 1), -2), (dict(K=0), -2),
    (dict(K=60, ldx=64), -2), (dict(K=(1 << 20) + 8), -2), (dict(act=5), -3), (dict(act=-1), -3), (dict(ot=2), -3),
    (dict(x=None), -1), (dict(W=None), -1), (dict(out=None), -1), (dict(ldx=56), -2), (dict(ldx=68), -2),
    (dict(ldw=68), -2), (dict(ldw=8), -2), (dict(ldx=(1 << 22) + 8), -2), (dict(x=ODD), -2), (dict(W=ODD), -2),
    (dict(ldo=9), -2), (dict(res=A, ldr=9), -2), (dict(T=0, x=None, W=None, out=None), 0),
])
def test_linear_refusals(kw, want):
    assert rc("moe_linear", LIN, **kw) == want
    assert want == 0 or ops.last_error()


def test_linear_refuses_a_small_workspace():
    # a few tiles of 7168 summands are split along K; up to 4 rows need no workspace
    n = ops.workspace_bytes("moe_linear_workspace", 100, 256, 7168)
    assert n > 0 and ops.workspace_bytes("moe_linear_workspace", 4, 256, 7168) == 0
    kw = dict(T=100, N=256, K=7168, ldx=7168, ldw=7168, ldo=256)
    assert rc("moe_linear", LIN, wsb=n - 1, **kw) == -4
    assert rc("moe_linear", LIN, ws=None, **kw) == -4


LINB = dict(dy=A, dt=0, pre=None, x=A, ldx=64, W=A, ldw=64, add=None, T=4, N=16, K=64, act=0, dx=A, dW=A, db=A, ws=A,
            wsb=BIG, s=None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), -2), (dict(N=0), -2), (dict(K=12), -2), (dict(act=7), -3), (dict(dt=3), -3), (dict(dy=None), -1),
    (dict(x=None), -1), (dict(W=None), -1), (dict(act=1), -1), (dict(dx=ODD), -2), (dict(dW=ODD), -2),
    (dict(add=ODD), -2), (dict(dy=ODD), -2), (dict(act=1, pre=ODD), -2), (dict(ldx=68), -2), (dict(ldw=32), -2),
    (dict(ws=None), -1), (dict(ws=ODD), -1), (dict(wsb=16), -4),
    (dict(T=0, dW=None, db=None, dy=None, x=None, W=None), 0),
])
def test_linear_backward_refusals(kw, want):
    assert rc("moe_linear_backward", LINB, **kw) == want


FFN = dict(x=A, ldx=64, W13=A, b13=None, W2=A, b2=None, res=None, T=4, d=64, f=128, act=2, h=A, y=A, save=0, gu=None,
           gs=None, ws=A, wsb=BIG, s=None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), -2), (dict(d=60), -2), (dict(f=4), -2), (dict(f=1 << 20), -2), (dict(act=9), -3), (dict(save=3), -3),
    (dict(save=2, f=120, gu=A, gs=A), -2), (dict(save=1), -1), (dict(save=2, gu=A), -1), (dict(x=None), -1),
    (dict(W13=None), -1), (dict(h=None), -1), (dict(W2=None), -1), (dict(ldx=32), -2), (dict(ldx=68), -2),
    (dict(x=ODD), -2), (dict(W13=ODD), -2), (dict(h=ODD), -2), (dict(y=ODD), -2), (dict(b13=ODD), -2),
    (dict(res=ODD), -2), (dict(save=1, gu=ODD), -2), (dict(T=0, x=None, h=None), 0),
])
def test_gated_ffn_refusals(kw, want):
    assert rc("moe_gated_ffn", FFN, **kw) == want


FFNB = dict(dy=A, x=A, ldx=64, W13=A, W2=A, save=1, gu=A, gs=None, add=None, T=4, d=64, f=128, act=2, dx=A, dW13=A,
            dW2=A, db13=None, db2=None, ws=A, wsb=BIG, s=None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), -2), (dict(save=0), -3), (dict(save=2), -1), (dict(dy=None), -1), (dict(gu=None), -1),
    (dict(x=None), -1), (dict(W13=None), -1), (dict(W2=None), -1), (dict(dx=ODD), -2), (dict(add=ODD), -2),
    (dict(dW2=ODD), -2), (dict(x=ODD), -2), (dict(ldx=63), -2), (dict(ws=None), -1), (dict(wsb=100), -4),
    (dict(T=0, dW13=None, dW2=None), 0),
])
def test_gated_ffn_backward_refusals(kw, want):
    assert rc("moe_gated_ffn_backward", FFNB, **kw) == want


@pytest.mark.parametrize("kw, want", [
    (dict(rows=-1), -2), (dict(cols=12), -2), (dict(cols=0), -2), (dict(src=None), -1), (dict(q=None), -1),
    (dict(s=None), -1), (dict(ld=120), -2), (dict(ld=132), -2), (dict(src=ODD), -2), (dict(q=ODD), -2),
    (dict(rows=1 << 30, cols=1 << 20, ld=1 << 20), -2), (dict(s=ODD), -2), (dict(rows=0, src=None), 0),
])
def test_act_save_refusals(kw, want):
    assert rc("moe_act_save", dict(src=A, ld=128, rows=4, cols=128, q=A, s=A, st=None), **kw) == want


@pytest.mark.parametrize("kw, want", [
    (dict(rows=-1), -2), (dict(cols=4), -2), (dict(q=None), -1), (dict(s=None), -1), (dict(dst=None), -1),
    (dict(dst=ODD), -2), (dict(rows=0, q=None), 0),
])
def test_act_restore_refusals(kw, want):
    assert rc("moe_act_restore", dict(q=A, s=A, rows=4, cols=128, dst=A, st=None), **kw) == want


def test_workspace_functions():
    n = ctypes.c_size_t(0)
    for fn in ("moe_linear_workspace", "moe_linear_backward_workspace", "moe_gated_ffn_workspace",
               "moe_gated_ffn_backward_workspace"):
        f = getattr(ops.lib(), fn)
        assert f(4, 64, 64, None) == -1
        assert f(4, 64, 63, ctypes.byref(n)) == -2
        assert f(-1, 64, 64, ctypes.byref(n)) == -2
        assert f(0, 64, 64, ctypes.byref(n)) == 0
        assert f(4, 64, 64, ctypes.byref(n)) == 0


def test_wrappers_refuse():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        ops.act_save(x)
    with pytest.raises(TypeError, match="expected"):
        ops.act_save(x.float())
    with pytest.raises(ValueError, match="adjacent"):
        ops.act_save(torch.zeros(128, 4, dtype=torch.bfloat16).t())
