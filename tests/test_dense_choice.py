"""CPU checks of which kernels the dense products take (256 compute units)."""

import ctypes
import os

import pytest

from moe_expert_layer_r3_amd import ops

pytestmark = pytest.mark.skipif(not os.path.exists(ops.LIB_PATH), reason="library not built")


def answer(name, *args):
    v = ctypes.c_int32(-1)
    ops._call(name, *args, ctypes.byref(v))
    return bool(v.value)


@pytest.mark.parametrize("T", [16384, 65536, 1 << 18, 1 << 20, 1 << 30])
@pytest.mark.parametrize("N, K", [(8, 8), (64, 64), (256, 64), (64, 1024), (256, 1024)])
def test_long_column_sums_are_not_grouped(T, N, K):
    """A column sum in the group walks all rows in one workgroup: without a
    weight gradient of the same length beside it that takes far longer than the
    sum's own two launches."""
    assert not answer("moe_linear_backward_grouped", T, N, K, 0, 0, 1, 0, 1)
    if K < 1024 or T > 16384:   # (f = 1024 over 16384 rows: about even)
        assert not answer("moe_gated_ffn_backward_grouped", T, N, K, 1, 0, 0, 1)


def test_small_gradients_are_grouped():
    for T in (16, 200, 1024):
        assert answer("moe_linear_backward_grouped", T, 64, 64, 0, 0, 1, 1, 1)
        assert answer("moe_linear_backward_grouped", T, 64, 64, 0, 0, 1, 0, 1)
        assert answer("moe_gated_ffn_backward_grouped", T, 64, 64, 1, 1, 1, 1)
        assert answer("moe_gated_ffn_backward_grouped", T, 64, 64, 1, 0, 0, 1)
    # dz is made first, and its chunks of rows are summed: at most 1024 rows
    assert answer("moe_linear_backward_grouped", 200, 64, 64, 1, 0, 1, 0, 1)
    # one gradient alone, or none, is no group
    for on in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 0, 0)):
        assert not answer("moe_linear_backward_grouped", 200, 64, 64, 0, 0, *on)
    assert not answer("moe_linear_backward_grouped", 0, 64, 64, 0, 0, 1, 1, 1)


def test_grouped_refusals():
    lib, v = ops.lib(), ctypes.c_int32(0)
    assert lib.moe_linear_backward_grouped(4, 64, 64, 0, 0, 1, 1, 1, None) == -1
    assert lib.moe_linear_backward_grouped(4, 64, 63, 0, 0, 1, 1, 1, ctypes.byref(v)) == -2
    assert lib.moe_gated_ffn_backward_grouped(4, 64, 64, 1, 1, 1, 1, None) == -1
    assert lib.moe_gated_ffn_backward_grouped(4, 60, 64, 1, 1, 1, 1, ctypes.byref(v)) == -2


def test_dense_kernel_answers():
    assert ops.dense_kernel(1, 256, 7168) == ("thin", 0)
    assert ops.dense_kernel(48, 256, 7168)[0] == "slab"
    assert ops.dense_kernel(4, 256, 64, "gated_int8")[0] == "slab"
    for product in ("forward", "gated", "gradient"):
        assert ops.dense_kernel(16384, 4096, 7168, product) == ("wide", 0)
    # the pieces' workspace is what the choice says
    for T, N, K in ((100, 256, 7168), (8192, 256, 7168), (203, 1001, 520), (1237, 776, 3080)):
        n = ops.workspace_bytes("moe_linear_workspace", T, N, K)
        assert n == ops.dense_kernel(T, N, K)[1] * T * ((N + 3) // 4 * 4) * 4


def test_dense_kernel_refusals():
    lib, a, b = ops.lib(), ctypes.c_int32(0), ctypes.c_int32(0)
    f = lambda *s, k=ctypes.byref(a), p=ctypes.byref(b): lib.moe_dense_kernel(*s, k, p)
    assert f(1, 1, 1, 0) == 0
    assert f(1, 1, 1, 0, k=None) == -1 and f(1, 1, 1, 0, p=None) == -1
    assert f(1, 1, 1, 4) == -3 and f(1, 1, 1, -1) == -3
    for s in ((0, 1, 1), (1, 0, 1), (1, 1, 0), ((1 << 30) + 1, 1, 1), (1, (1 << 20) + 1, 1), (1, 1, (1 << 30) + 1)):
        assert f(*s, 0) == -2
