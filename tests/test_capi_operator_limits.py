"""Sizes whose launch would exceed the 2**32 threads that a grid dimension may
have: refused on the host with a message, nothing launched (no GPU needed)."""
import ctypes

import pytest

from test_capi_exports import _lib

v = ctypes.c_void_p
i64, i32, size = ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
P, O = v(4096), v(0)         # an aligned address that no refused call touches
BIG = size(1 << 62)


def refused(name, *args):
    L = _lib()
    L.moe4_last_error.restype = ctypes.c_char_p
    f = getattr(L, name)
    f.restype = ctypes.c_int
    assert f(*args) == -1
    msg = L.moe4_last_error().decode()
    assert name in msg
    return msg


def test_balance_loss_and_gradient():
    for T in ((1 << 28) - 63, 1 << 28, (1 << 31) - 1):
        assert "2^28" in refused("moe_balance_loss", P, O, P, O, O, i32(1), i64(T), i32(2), i32(1), P, P, P, P, P, BIG, O)
        assert "2^28" in refused("moe_balance_loss_backward", P, P, O, P, P, O, O, i32(1), i64(T), i32(2), i32(1), O, P, O)


@pytest.mark.parametrize("copies", [1, 8])
def test_quant_of_no_rows_with_an_empty_map(copies):
    """An empty map's pointer is NULL: nothing to do, whatever copies says."""
    f = _lib().mxfp4_quant
    f.restype = ctypes.c_int
    assert f(O, 0, i64(0), i64(64), O, i32(copies), i64(0), 0, O, O, O) == 0


@pytest.mark.parametrize("name,args", [
    ("mxfp4_quant", (P, 0, i64(1 << 32), i64(32), O, i32(1), i64(1 << 32), 0, P, P, O)),
    ("mxfp4_dequant", (P, P, i64(1 << 30), i64(32), P, 0, O)),
    ("mxfp8_requant_mx4_sr_T", (P, P, i64(1 << 30), i64(32), P, P, i32(1), i64(1 << 31), ctypes.c_uint64(1), ctypes.c_uint32(0), 0, P, P, O)),
    ("moe_grouped_gemm_mx4", (P, P, P, P, P, i32(1 << 24), i64(1 << 24), i64(32), i64(32), P, 0, O)),
    ("moe_unpermute_sum_router_dense", (P, P, i64(1 << 30), i32(1), i64(4), P, i32(1), P, P, O)),
    ("moe_unpermute_sum_router_dense", (P, P, i64(((1 << 24) - 3) * 64), i32(1), i64(4), P, i32(1), P, P, O)),   # (the grid is a multiple of 8)
    ("moe_router_wgrad_dense", (P, P, i64(64), i32(1 << 19), i64(1 << 19), P, O, size(0), O))])
def test_too_large(name, args):
    assert "too large" in refused(name, *args)
