"""Refusals of the MXFP4, balance-loss and dense router calls: every bad size,
type, pointer or workspace is an error code with a message, and nothing is
enqueued (host checks: this runs without a GPU)."""
import ctypes

import pytest

from test_capi_exports import _lib

v = ctypes.c_void_p
i64, i32, size = ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
P = v(4096)          # an aligned address that no refused call touches
EINVAL, EALIGN, EWS = -1, -2, -3


def call(name, *args):
    f = getattr(_lib(), name)
    f.restype = ctypes.c_int
    return f(*args)


def quant(x=P, dt=0, rows=4, cols=64, omap=v(0), copies=1, out_rows=4, pre=0, codes=P, sf=P):
    return call("mxfp4_quant", x, dt, i64(rows), i64(cols), omap, i32(copies), i64(out_rows), pre, codes, sf, v(0))


@pytest.mark.parametrize("kw,rc", [
    (dict(cols=48), EINVAL), (dict(cols=0), EINVAL), (dict(rows=-1, out_rows=-1), EINVAL), (dict(dt=2), EINVAL),
    (dict(pre=1, dt=1), EINVAL), (dict(pre=2), EINVAL), (dict(copies=2), EINVAL), (dict(out_rows=5), EINVAL),
    (dict(omap=P, copies=0), EINVAL), (dict(omap=P, copies=1 << 30, out_rows=8), EINVAL),
    (dict(x=v(0)), EINVAL), (dict(codes=v(0)), EINVAL), (dict(sf=v(0)), EINVAL),
    (dict(x=v(4104)), EALIGN), (dict(codes=v(4100)), EALIGN), (dict(rows=0, out_rows=0, x=v(0)), 0)])
def test_mxfp4_quant_refusals(kw, rc):
    assert quant(**kw) == rc


@pytest.mark.parametrize("kw,rc", [(dict(cols=40), EINVAL), (dict(dt=3), EINVAL), (dict(out=v(0)), EINVAL),
                                   (dict(out=v(4097)), EALIGN), (dict(rows=0, out=v(0)), 0)])
def test_mxfp4_dequant_refusals(kw, rc):
    a = dict(rows=4, cols=64, out=P, dt=1, **{})
    a.update(kw)
    assert call("mxfp4_dequant", P, P, i64(a["rows"]), i64(a["cols"]), a["out"], a["dt"], v(0)) == rc


@pytest.mark.parametrize("kw,rc", [(dict(cols=33), EINVAL), (dict(G=0), EINVAL), (dict(mpr=40), EINVAL), (dict(lay=2), EINVAL),
                                   (dict(off=v(0)), EINVAL), (dict(codes=v(4104)), EALIGN), (dict(mpr=0), 0)])
def test_requant_mx4_refusals(kw, rc):
    a = dict(cols=64, G=1, mpr=64, lay=0, off=P, codes=P)
    a.update(kw)
    assert call("mxfp8_requant_mx4_sr_T", a["codes"], P, i64(40), i64(a["cols"]), a["off"], P, i32(a["G"]), i64(a["mpr"]),
                ctypes.c_uint64(1), ctypes.c_uint32(0), a["lay"], P, P, v(0)) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(K=48), EINVAL), (dict(N=40), EINVAL), (dict(E=0), EINVAL), (dict(M=-1), EINVAL), (dict(M=1 << 31), EINVAL), (dict(dt=2), EINVAL),
    (dict(N=1 << 17, K=1 << 15), EINVAL), (dict(c=v(0)), EINVAL), (dict(off=v(0)), EINVAL), (dict(c=v(4104)), EALIGN),
    (dict(a=v(4100)), EALIGN), (dict(M=0, a=v(0), c=v(0)), 0)])
def test_gemm_mx4_refusals(kw, rc):
    a = dict(E=2, M=8, N=64, K=64, a=P, off=P, c=P, dt=0)
    a.update(kw)
    assert call("moe_grouped_gemm_mx4", a["a"], P, P, P, a["off"], i32(a["E"]), i64(a["M"]), i64(a["N"]), i64(a["K"]), a["c"],
                a["dt"], v(0)) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(k=0), EINVAL), (dict(k=17), EINVAL), (dict(k=9, E=8), EINVAL), (dict(E=1025), EINVAL), (dict(T=-1), EINVAL),
    (dict(T=1 << 30), EINVAL), (dict(S=0), EINVAL), (dict(S=2), EINVAL), (dict(z=v(0)), EINVAL), (dict(loss=v(0)), EINVAL),
    (dict(nbytes=16), EWS), (dict(ws=v(0)), EWS), (dict(ws=v(4100)), EALIGN)])
def test_balance_loss_refusals(kw, rc):
    a = dict(T=8, E=64, k=8, S=1, z=P, loss=P, ws=P, nbytes=1 << 20)
    a.update(kw)
    assert call("moe_balance_loss", a["z"], v(0), P, v(0), v(0), i32(a["S"]), i64(a["T"]), i32(a["E"]), i32(a["k"]), a["loss"], P,
                P, P, a["ws"], size(a["nbytes"]), v(0)) == rc


@pytest.mark.parametrize("kw,rc", [(dict(k=0), EINVAL), (dict(E=2000), EINVAL), (dict(S=3), EINVAL), (dict(T=1 << 31), EINVAL),
                                   (dict(out=v(0)), EINVAL), (dict(T=0, out=v(0)), 0)])
def test_balance_backward_refusals(kw, rc):
    a = dict(T=8, E=64, k=8, S=1, out=P)
    a.update(kw)
    assert call("moe_balance_loss_backward", P, P, v(0), P, P, v(0), v(0), i32(a["S"]), i64(a["T"]), i32(a["E"]), i32(a["k"]),
                v(0), a["out"], v(0)) == rc


@pytest.mark.parametrize("kw,rc", [(dict(k=0), EINVAL), (dict(k=17), EINVAL), (dict(E=0), EINVAL), (dict(d=66), EINVAL), (dict(dxp=v(0)), EINVAL),
                                   (dict(T=1 << 30), EINVAL), (dict(dxp=v(4104)), EALIGN), (dict(T=0, dxp=v(0)), 0)])
def test_unpermute_router_dense_refusals(kw, rc):
    a = dict(T=8, k=2, d=64, E=4, dxp=P)
    a.update(kw)
    assert call("moe_unpermute_sum_router_dense", a["dxp"], P, i64(a["T"]), i32(a["k"]), i64(a["d"]), P, i32(a["E"]), P, P,
                v(0)) == rc


@pytest.mark.parametrize("kw,rc", [(dict(E=0), EINVAL), (dict(d=30), EINVAL), (dict(T=-1), EINVAL), (dict(dw=v(0)), EINVAL), (dict(dw=v(4100)), EALIGN),
                                   (dict(T=100000, nbytes=64), EWS), (dict(T=100000, ws=v(0)), EWS)])
def test_router_wgrad_dense_refusals(kw, rc):
    a = dict(T=8, E=4, d=64, dw=P, ws=P, nbytes=1 << 40)
    a.update(kw)
    assert call("moe_router_wgrad_dense", P, P, i64(a["T"]), i32(a["E"]), i64(a["d"]), a["dw"], a["ws"], size(a["nbytes"]),
                v(0)) == rc


@pytest.mark.parametrize("kw", [dict(E=1 << 20), dict(d=1 << 28)])
def test_router_dense_sizes_past_a_descriptor(kw):
    a = dict(E=4, d=64)
    a.update(kw)
    assert call("moe_unpermute_sum_router_dense", P, P, i64(8), i32(2), i64(a["d"]), P, i32(a["E"]), P, P, v(0)) == EINVAL
    assert call("moe_router_wgrad_dense", P, P, i64(8), i32(a["E"]), i64(a["d"]), P, P, size(1 << 40), v(0)) == EINVAL


def test_workspace_queries():
    L = _lib()
    L.moe_balance_loss_ws_bytes.restype = L.moe_router_wgrad_dense_ws_bytes.restype = size
    assert L.moe_balance_loss_ws_bytes(i64(-1), i32(4), i32(1)) == 0
    # at least a partial row of E sums and counts per segment
    assert L.moe_balance_loss_ws_bytes(i64(1000), i32(64), i32(37)) >= 37 * 64 * 8
    assert L.moe_router_wgrad_dense_ws_bytes(i64(8), i32(4), i64(64)) == 0


def test_binding_refusals():
    """The Python binding refuses CPU tensors, wrong types and wrong shapes before the library sees a pointer."""
    import torch
    import precision_moe_numerics_quant_amd as m4
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        m4.mxfp4_quant(x)
    with pytest.raises(ValueError, match="bf16 or float32"):
        m4.mxfp4_quant(x.half())
    with pytest.raises(ValueError, match="out_dtype"):
        m4.mxfp4_dequant(x, x, torch.float16)
    with pytest.raises(ValueError, match="out_dtype"):
        m4.moe_grouped_gemm_mx4(x, x, x, x, x, torch.float16)
    with pytest.raises(ValueError):
        m4.moe_balance_loss(torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32))
    with pytest.raises(ValueError):
        m4.moe_router_wgrad_dense(x, torch.zeros((4, 8)))
