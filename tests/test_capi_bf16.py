"""Refusals of the BF16 products and the dropout calls: bad sizes, types, pointers and
maps are error codes with a message and nothing is enqueued (host checks: no GPU needed)."""
import ctypes

import pytest

from test_capi_exports import _lib

v = ctypes.c_void_p
i64, i32, f32, f64 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_double
P, O = v(4096), v(0)         # an aligned address that no refused call touches; NULL
EINVAL, EALIGN, EWS = -1, -2, -3


def call(name, *args):
    L = _lib()
    L.moe4_last_error.restype = ctypes.c_char_p
    f = getattr(L, name)
    f.restype = ctypes.c_int
    rc = f(*args)
    assert rc == 0 or name.encode() in L.moe4_last_error()
    return rc


DEF = dict(a=P, rows=8, map=O, div=1, w=P, bias=O, scale=O, off=P, E=2, M=8, N=64, K=64, act=0, res=O, c=P, dt=0, aux=O, pre=O)


def gemm(d):
    return call("moe_grouped_gemm_bf16", d["a"], i64(d["rows"]), d["map"], i32(d["div"]), d["w"], d["bias"], d["off"], i32(d["E"]), i64(d["M"]),
                i64(d["N"]), i64(d["K"]), d["act"], d["res"], d["c"], d["dt"], d["aux"], O)


def gated(d):
    return call("moe_gated_gemm_bf16", d["a"], i64(d["rows"]), d["map"], i32(d["div"]), d["w"], d["bias"], d["off"], i32(d["E"]), i64(d["M"]),
                i64(d["N"]), i64(d["K"]), d["act"], d["c"], d["aux"], O)


def dgrad(d):
    return call("moe_grouped_gemm_bf16_dgrad", d["a"], i64(d["rows"]), d["map"], i32(d["div"]), d["scale"], d["w"], d["off"], i32(d["E"]),
                i64(d["M"]), i64(d["N"]), i64(d["K"]), d["act"], d["pre"], d["res"], d["c"], d["dt"], d["aux"], O)


def gated_dgrad(d):
    return call("moe_gated_gemm_bf16_dgrad", d["a"], i64(d["rows"]), d["map"], i32(d["div"]), d["scale"], d["w"], d["off"], i32(d["E"]),
                i64(d["M"]), i64(d["N"]), i64(d["K"]), d["act"], d["pre"], d["c"], d["aux"], O)


@pytest.mark.parametrize("f", [gemm, gated, dgrad, gated_dgrad])
@pytest.mark.parametrize("kw,rc", [
    (dict(N=60), EINVAL), (dict(K=20), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(E=0), EINVAL), (dict(E=4097), EINVAL),
    (dict(M=-1, rows=-1), EINVAL), (dict(M=1 << 31, rows=1 << 31), EINVAL), (dict(N=1 << 20), EINVAL), (dict(N=1 << 17, K=1 << 12), EINVAL),
    (dict(rows=7), EINVAL), (dict(map=P, div=0), EINVAL), (dict(map=P, div=-3), EINVAL), (dict(map=P, div=2, rows=0), EINVAL),
    (dict(map=P, div=2, rows=1 << 24), EINVAL), (dict(act=3), EINVAL), (dict(act=-1), EINVAL), (dict(off=O), EINVAL), (dict(a=O), EINVAL),
    (dict(w=O), EINVAL), (dict(c=O), EINVAL), (dict(a=v(4104)), EALIGN), (dict(w=v(4098)), EALIGN), (dict(c=v(4100)), EALIGN),
    (dict(aux=v(4104), pre=P), EALIGN), (dict(map=v(4098)), EALIGN), (dict(M=0, rows=0, a=O, w=O, c=O), 0)])
def test_product_refusals(f, kw, rc):
    assert f({**DEF, "pre": P if f is gated_dgrad else O, **kw}) == rc


@pytest.mark.parametrize("kw,rc", [(dict(dt=2), EINVAL), (dict(res=v(4104)), EALIGN), (dict(bias=v(4100)), EALIGN)])
def test_gemm_refusals(kw, rc):
    assert gemm({**DEF, **kw}) == rc


@pytest.mark.parametrize("kw,rc", [(dict(dt=-1), EINVAL), (dict(act=1), EINVAL), (dict(aux=P), EINVAL), (dict(scale=v(4098)), EALIGN),
                                   (dict(pre=v(4104)), EALIGN), (dict(res=v(4104)), EALIGN)])
def test_dgrad_refusals(kw, rc):
    assert dgrad({**DEF, **kw}) == rc


@pytest.mark.parametrize("act", [0, 1, 2])
def test_dgrad_of_no_rows(act):
    """Empty tensors have no address: pre may be NULL where there are no rows, with an activation too."""
    none = dict(M=0, rows=0, a=O, w=O, c=O, pre=O, act=act)
    assert dgrad({**DEF, **none}) == 0 and gated_dgrad({**DEF, **none}) == 0


def test_gated_dgrad_needs_gu():
    assert gated_dgrad({**DEF, "pre": O}) == EINVAL


W = dict(dy=P, dyr=8, dym=O, a=P, ar=8, am=O, div=1, off=P, E=2, M=8, N=64, K=64, dw=P, beta=0.0, flags=0, sc=O, db=O, ws=O, wsb=0)


def wgrad(**kw):
    d = {**W, **kw}
    return call("moe_grouped_gemm_bf16_wgrad", d["dy"], i64(d["dyr"]), d["dym"], d["a"], i64(d["ar"]), d["am"], i32(d["div"]), d["off"],
                i32(d["E"]), i64(d["M"]), i64(d["N"]), i64(d["K"]), d["dw"], f32(d["beta"]), d["flags"], d["sc"], d["db"], d["ws"],
                ctypes.c_size_t(d["wsb"]), O)


@pytest.mark.parametrize("kw,rc", [
    (dict(N=12), EINVAL), (dict(K=4), EINVAL), (dict(E=0), EINVAL), (dict(E=5000), EINVAL), (dict(M=-8, dyr=-8, ar=-8), EINVAL), (dict(dyr=9), EINVAL),
    (dict(ar=9), EINVAL), (dict(N=1 << 17, K=1 << 12), EINVAL), (dict(beta=0.5), EINVAL), (dict(flags=2), EINVAL), (dict(dw=O), EINVAL), (dict(off=O), EINVAL),
    (dict(dy=O), EINVAL), (dict(a=O), EINVAL), (dict(dym=P, div=0), EINVAL), (dict(am=P, ar=0), EINVAL), (dict(dym=P, dyr=1 << 24), EINVAL),
    (dict(am=P, ar=1 << 24), EINVAL), (dict(sc=P), EINVAL), (dict(dw=v(4104)), EALIGN), (dict(db=v(4104)), EALIGN), (dict(dy=v(4104)), EALIGN),
    (dict(am=v(4098)), EALIGN), (dict(M=4096, dyr=4096, ar=4096), EWS), (dict(M=4096, dyr=4096, ar=4096, ws=P, wsb=1000), EWS),
    (dict(M=4096, dyr=4096, ar=4096, ws=v(4104), wsb=1 << 20), EALIGN)])
def test_wgrad_refusals(kw, rc):
    assert wgrad(**kw) == rc


@pytest.mark.parametrize("E,M,N,K", [(1, 8, 1 << 39, 1 << 40), (128, 8, 1 << 62, 8), (2, 4096, 1 << 20, 64), (2, 4096, 1 << 17, 1 << 12), (2049, 8, 64, 64),
                                     (0, 8, 64, 64), (2, -1, 64, 64), (2, 1 << 31, 64, 64), (2, 4096, 0, 64), (2, 4096, 64, -8), (2, 4096, 60, 64)])
def test_wgrad_workspace_of_refused_sizes(E, M, N, K):
    """0 for what the call refuses, however large (in a process of its own: the sizes' products may wrap to a divisor of 0)."""
    import subprocess
    import sys
    from test_capi_exports import LIB
    _lib()
    code = ("import ctypes; f = ctypes.CDLL(%r).moe_grouped_gemm_bf16_wgrad_ws_bytes; f.restype = ctypes.c_size_t; "
            "print(f(ctypes.c_int32(%d), ctypes.c_int64(%d), ctypes.c_int64(%d), ctypes.c_int64(%d)))" % (LIB, E, M, N, K))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "0", (r.returncode, r.stdout, r.stderr[-300:])


def test_wgrad_workspace_of_served_sizes():
    """Few experts with many rows need one, one that would not pay for its join does not."""
    f = _lib().moe_grouped_gemm_bf16_wgrad_ws_bytes
    f.restype = ctypes.c_size_t
    size = lambda E, M, N, K: f(i32(E), i64(M), i64(N), i64(K))  # noqa: E731
    assert size(1, 16384, 1536, 4096) >= 2 * 1536 * 4096 * 4 and size(2048, 16384, 1536, 4096) == 0 and size(1, 8, 64, 64) == 0


def drop(yp=P, T=8, k=2, d=64, p=0.1, res=O, y=P):
    return call("moe_combine_dropout", yp, P, P, i64(T), i32(k), i64(d), f64(p), ctypes.c_uint64(1), ctypes.c_uint32(0), res, y, O)


@pytest.mark.parametrize("kw,rc", [
    (dict(k=0), EINVAL), (dict(k=17), EINVAL), (dict(d=66), EINVAL), (dict(d=0), EINVAL), (dict(T=-1), EINVAL), (dict(p=-0.1), EINVAL), (dict(p=1.1), EINVAL),
    (dict(p=float("nan")), EINVAL), (dict(T=1 << 30), EINVAL), (dict(T=1 << 24, d=1 << 20), EINVAL), (dict(yp=O), EINVAL), (dict(y=O), EINVAL),
    (dict(yp=v(4104)), EALIGN), (dict(res=v(4104)), EALIGN), (dict(T=0, yp=O, y=O), 0)])
def test_combine_dropout_refusals(kw, rc):
    assert drop(**kw) == rc


@pytest.mark.parametrize("kw,rc", [(dict(d=2), EINVAL), (dict(T=-1), EINVAL), (dict(p=2.0), EINVAL), (dict(p=float("nan")), EINVAL),
                                   (dict(T=1 << 30, d=1 << 10), EINVAL), (dict(dy=O), EINVAL), (dict(dx=v(4104)), EALIGN), (dict(T=0, dy=O), 0)])
def test_dropout_backward_refusals(kw, rc):
    d = {**dict(dy=P, T=8, d=64, p=0.5, dx=P), **kw}
    assert call("moe_dropout_backward", d["dy"], i64(d["T"]), i64(d["d"]), f64(d["p"]), ctypes.c_uint64(1), ctypes.c_uint32(0), d["dx"], O) == rc


def test_binding_refusals():
    """The Python binding refuses CPU tensors and wrong types before the library sees a pointer."""
    import torch
    import precision_moe_numerics_quant_amd as m4
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((2, 64, 64), dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    for call_ in (lambda: m4.moe_grouped_gemm_bf16(x, w, off), lambda: m4.moe_gated_gemm_bf16(x, w.view(1, 2, 64, 64), off),
                  lambda: m4.moe_grouped_gemm_bf16_dgrad(x, w, off), lambda: m4.moe_gated_gemm_bf16_dgrad(x, w, x, off),
                  lambda: m4.moe_grouped_gemm_bf16_wgrad(x, x, off), lambda: m4.moe_dropout_backward(x, 0.1)):
        with pytest.raises(ValueError, match="GPU"):
            call_()
    with pytest.raises(ValueError, match="out_dtype"):
        m4.moe_grouped_gemm_bf16(x, w, off, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out_dtype"):
        m4.moe_grouped_gemm_bf16_dgrad(x, w, off, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="needs a map"):
        m4.moe_grouped_gemm_bf16_wgrad(x, x, off, map_div=2)
