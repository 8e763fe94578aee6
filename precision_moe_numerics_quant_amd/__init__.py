"""MI355X-native NVFP4-forward / MXFP8-backward MoE expert layer.

Thin Python binding of ``libmoe4.so`` (C ABI in ``include/moe4.h``): each
function checks tensor devices, dtypes and shapes, allocates outputs with
torch, passes raw device pointers and torch's current HIP stream, and raises
on a non-zero return code.  Every step of the computation runs in the HIP
kernels; there is no CPU or PyTorch fallback: if the library is missing the
functions raise.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe4.so")

BF16, F32 = 0, 1
NVFP4_6, NVFP4_4OVER6 = 6, 46
PRE_NONE, PRE_SILU, PRE_SILU_AMAX = 0, 1, 2
EUNSUPPORTED = -5
EDEVICE = -6
RNE, SR = 0, 1
ACT_NONE, ACT_SILU, ACT_GELU = 0, 1, 2
SF_ROWS, SF_BLOCKS = 0, 1   # group-major scale arrangement: [C][P_g/32] or [P_g/32][C]

_c_void_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_int = ctypes.c_int
_u64 = ctypes.c_uint64
_u32 = ctypes.c_uint32
_f32 = ctypes.c_float
_f64 = ctypes.c_double
_size = ctypes.c_size_t

_SIGS = {
    "moe4_last_error": (ctypes.c_char_p, []),
    "moe4_version": (ctypes.c_char_p, []),
    "nvfp4_quant_46": (_int, [_c_void_p, _int, _i64, _i64, _c_void_p, _i32, _int, _int, _c_void_p, _c_void_p,
                              _c_void_p, _c_void_p, _size, _c_void_p]),
    "nvfp4_quant_46_ws_bytes": (_size, [_i32]),
    "nvfp4_quant_46_noalloc": (_int, [_c_void_p, _int, _i64, _i64, _c_void_p, _i32, _int, _int, _c_void_p,
                                      _c_void_p, _c_void_p, _c_void_p]),
    "nvfp4_quant_requant_T": (_int, [_c_void_p, _i64, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _u64, _u32,
                                     _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p]),
    "nvfp4_quant_requant_T_ws_bytes": (_size, [_i32]),
    "nvfp4_dequant": (_int, [_c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _i32, _i64, _i64, _c_void_p,
                             _c_void_p]),
    "mxfp8_requant_sr_T": (_int, [_c_void_p, _c_void_p, _c_void_p, _int, _i64, _i64, _c_void_p, _c_void_p, _i32,
                                  _i64, _u64, _u32, _int, _c_void_p, _c_void_p, _c_void_p]),
    "mxfp8_requant_mx_sr_T": (_int, [_c_void_p, _c_void_p, _i64, _i64, _c_void_p, _c_void_p, _i32, _i64, _u64,
                                     _u32, _int, _c_void_p, _c_void_p, _c_void_p]),
    "moe_grouped_gemm_mx": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i64, _i64,
                                   _c_void_p, _int, _c_void_p]),
    "mxfp8_quant": (_int, [_c_void_p, _int, _i64, _i64, _c_void_p, _i32, _c_void_p, _c_void_p, _int, _int,
                           _c_void_p, _c_void_p, _i32, _i64, _int, _u64, _u32, _c_void_p, _c_void_p, _c_void_p]),
    "mxfp8_quant_rows_T": (_int, [_c_void_p, _int, _i64, _i64, _c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p,
                                  _c_void_p, _i32, _i64, _int, _u64, _u32, _int, _c_void_p, _c_void_p, _c_void_p,
                                  _c_void_p, _c_void_p]),
    "moe_route_backward": (_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i32, _c_void_p, _c_void_p]),
    "moe_dgates": (_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i64, _c_void_p, _c_void_p]),
    "moe4_debug_check": (_int, [_c_void_p]),
    "moe4_debug_force_wait_timeout": (_int, [_int]),
    "moe_route_topk": (_int, [_c_void_p, _c_void_p, _i64, _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                              _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p]),
    "moe_route_topk_ws_bytes": (_size, [_i64, _i32, _i32]),
    "moe_gather_rows": (_int, [_c_void_p, _c_void_p, _i64, _i64, _c_void_p, _i32, _i64, _c_void_p, _c_void_p,
                               _c_void_p]),
    "moe_grouped_gemm_fwd": (_int, [_c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _i32, _i64, _i64, _i64, _c_void_p, _int, _c_void_p]),
    "moe_grouped_gemm_bwd_dgrad": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i64,
                                          _i64, _c_void_p, _c_void_p]),
    "moe_grouped_gemm_bwd_wgrad": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i64,
                                          _c_void_p, _f32, _int, _c_void_p]),
    "moe_grouped_gemm_bwd": (_int, [_c_void_p] * 10 + [_i32, _i64, _i64, _i64, _c_void_p, _c_void_p, _f32, _int,
                                                       _c_void_p]),
    "moe_combine": (_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i64, _c_void_p, _c_void_p]),
    "moe_unpermute_sum": (_int, [_c_void_p, _c_void_p, _i64, _i32, _i64, _c_void_p, _c_void_p]),
    "moe_silu_eval": (_int, [_c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p]),
    "moe_router_logits": (_int, [_c_void_p, _c_void_p, _i64, _i32, _i64, _c_void_p, _c_void_p]),
    "moe_unpermute_sum_router": (_int, [_c_void_p, _c_void_p, _i64, _i32, _i64, _c_void_p, _c_void_p, _i32, _c_void_p,
                                        _c_void_p, _c_void_p]),
    "moe_router_wgrad": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i32, _i64, _c_void_p,
                                _c_void_p, _size, _c_void_p]),
    "moe_router_wgrad_ws_bytes": (_size, [_i64, _i32, _i32, _i64]),
    "mxfp8_quant_requant_T": (_int, [_c_void_p, _i64, _i64, _i32, _u64, _u32, _c_void_p, _c_void_p, _c_void_p,
                                     _c_void_p, _c_void_p]),
    "moe_grouped_gemm_fwd_silu_amax": (_int, [_c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p, _c_void_p,
                                              _c_void_p, _i32, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p]),
    "moe_hmx8_quant": (_int, [_c_void_p, _i64, _i64, _c_void_p, _c_void_p, _c_void_p]),
    "moe_hmx8_dequant": (_int, [_c_void_p, _c_void_p, _i64, _i64, _c_void_p, _c_void_p]),
    "moe_combine_hmx8": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i64, _c_void_p,
                                _c_void_p]),
    "mxfp4_quant": (_int, [_c_void_p, _int, _i64, _i64, _c_void_p, _i32, _i64, _int, _c_void_p, _c_void_p, _c_void_p]),
    "mxfp4_dequant": (_int, [_c_void_p, _c_void_p, _i64, _i64, _c_void_p, _int, _c_void_p]),
    "mxfp8_requant_mx4_sr_T": (_int, [_c_void_p, _c_void_p, _i64, _i64, _c_void_p, _c_void_p, _i32, _i64, _u64,
                                      _u32, _int, _c_void_p, _c_void_p, _c_void_p]),
    "moe_grouped_gemm_mx4": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i64, _i64,
                                    _c_void_p, _int, _c_void_p]),
    "moe_balance_loss": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i32, _i32,
                                _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p]),
    "moe_balance_loss_ws_bytes": (_size, [_i64, _i32, _i32]),
    "moe_balance_loss_backward": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                         _i32, _i64, _i32, _i32, _c_void_p, _c_void_p, _c_void_p]),
    "moe_unpermute_sum_router_dense": (_int, [_c_void_p, _c_void_p, _i64, _i32, _i64, _c_void_p, _i32, _c_void_p,
                                              _c_void_p, _c_void_p]),
    "moe_router_wgrad_dense": (_int, [_c_void_p, _c_void_p, _i64, _i32, _i64, _c_void_p, _c_void_p, _size, _c_void_p]),
    "moe_router_wgrad_dense_ws_bytes": (_size, [_i64, _i32, _i64]),
    "moe_grouped_gemm_bf16": (_int, [_c_void_p, _i64, _c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i64,
                                     _i64, _int, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p]),
    "moe_gated_gemm_bf16": (_int, [_c_void_p, _i64, _c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i64,
                                   _i64, _int, _c_void_p, _c_void_p, _c_void_p]),
    "moe_grouped_gemm_bf16_dgrad": (_int, [_c_void_p, _i64, _c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _i32, _i64,
                                           _i64, _i64, _int, _c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p]),
    "moe_gated_gemm_bf16_dgrad": (_int, [_c_void_p, _i64, _c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _i32, _i64,
                                         _i64, _i64, _int, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "moe_grouped_gemm_bf16_wgrad": (_int, [_c_void_p, _i64, _c_void_p, _c_void_p, _i64, _c_void_p, _i32, _c_void_p, _i32,
                                           _i64, _i64, _i64, _c_void_p, _f32, _int, _c_void_p, _c_void_p, _c_void_p, _size,
                                           _c_void_p]),
    "moe_grouped_gemm_bf16_wgrad_ws_bytes": (_size, [_i32, _i64, _i64, _i64]),
    "moe_combine_dropout": (_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i64, _f64, _u64, _u32, _c_void_p,
                                   _c_void_p, _c_void_p]),
    "moe_dropout_backward": (_int, [_c_void_p, _i64, _i64, _f64, _u64, _u32, _c_void_p, _c_void_p]),
    "moe_grouped_gemm_fwd_hmx8": (_int, [_c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p, _c_void_p,
                                         _c_void_p, _i32, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p,
                                         _c_void_p]),
}

EXPORTS = tuple(_SIGS)
_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m precision_moe_numerics_quant_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


class Moe4Error(RuntimeError):
    pass


class Moe4Unsupported(Moe4Error):
    """The call does not support this shape or kernel choice (nothing was launched)."""


class Moe4DeviceError(Moe4Error):
    """moe4_debug_check found a device-side error report (a clamped index or a
    bounded wait that gave up)."""


def _check(rc, name):
    if rc != 0:
        msg = lib().moe4_last_error().decode(errors="replace")
        cls = {EUNSUPPORTED: Moe4Unsupported, EDEVICE: Moe4DeviceError}.get(rc, Moe4Error)
        raise cls(f"{name} failed ({rc}): {msg}")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev(t, dtype, name):
    if not (t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor on the GPU, got {t.dtype} on {t.device}")
    return t


def _empty(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


def _ws(nbytes, like):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=like.device)


def _arg(t, dtype, shape, name, like=None):
    """Check a tensor argument of the calls below: dtype, shape (None: any size
    there), contiguous, on the GPU, and on like's device."""
    _dev(t, dtype, name)
    s = t.shape
    if s != shape and (len(s) != len(shape) or any(w is not None and g != w for g, w in zip(s, shape))):
        raise ValueError(f"{name}: expected shape {tuple(shape)} (None: any), got {tuple(s)}")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name}: on {t.device}, the call's other tensors on {like.device}")
    return t


def _raw_stream(index):
    """hipStream_t of the current stream of device index."""
    return torch.cuda.current_stream(index).cuda_stream


# the same without making a Stream object (2 us of a call that takes 10)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _run(name, like, *args):
    """Call the library on like's device, on that device's current stream
    (tensors among the arguments as their pointers)."""
    args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    i = like.device.index
    if i == torch.cuda.current_device():
        rc = getattr(lib(), name)(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            rc = getattr(lib(), name)(*args, _raw_stream(i))
    if rc:
        _check(rc, name)


def pad32(n):
    return (int(n) + 31) // 32 * 32


def max_padded_rows(rows, n_groups):
    """Upper bound of the padded row count of a grouped transposed layout."""
    return pad32(rows + 31 * n_groups)


# --------------------------------------------------------------------- NVFP4

def nvfp4_quant_46(x, mode=NVFP4_4OVER6, group_row_off=None, pre_op=PRE_NONE, ws=None):
    """NVFP4 of x [R, C] (bf16 or float32) -> (codes [R, C/2] u8, sf [R, C/16] u8, ts [G] f32).
    ws: the workspace (uint8 tensor); with PRE_SILU_AMAX it must hold the group amax
    words written by moe_grouped_gemm_fwd_silu_amax."""
    dt = {torch.bfloat16: BF16, torch.float32: F32}.get(x.dtype)
    if dt is None:
        raise ValueError("nvfp4_quant_46: x must be bf16 or float32")
    _dev(x, x.dtype, "x")
    R, C = x.shape
    G = 1 if group_row_off is None else group_row_off.numel() - 1
    if group_row_off is not None:
        _dev(group_row_off, torch.int32, "group_row_off")
    codes = _empty((R, C // 2), torch.uint8, x)
    sf = _empty((R, C // 16), torch.uint8, x)
    ts = _empty((G,), torch.float32, x)
    if ws is None:
        ws = _ws(lib().nvfp4_quant_46_ws_bytes(G), x)
    rc = lib().nvfp4_quant_46(_p(x), dt, R, C, _p(group_row_off), G, mode, pre_op, _p(codes), _p(sf), _p(ts),
                              _p(ws), ws.numel(), _stream())
    _check(rc, "nvfp4_quant_46")
    return codes, sf, ts


def nvfp4_quant_46_noalloc(x, mode=NVFP4_4OVER6, group_row_off=None, pre_op=PRE_NONE, out=None):
    """nvfp4_quant_46 with the library's static scratch instead of a workspace.
    out: optional (codes, sf, ts) tensors to write into (nothing is allocated
    then); otherwise they are allocated here, outside the library call."""
    dt = {torch.bfloat16: BF16, torch.float32: F32}.get(x.dtype)
    if dt is None:
        raise ValueError("nvfp4_quant_46_noalloc: x must be bf16 or float32")
    _dev(x, x.dtype, "x")
    R, C = x.shape
    G = 1 if group_row_off is None else group_row_off.numel() - 1
    if group_row_off is not None:
        _dev(group_row_off, torch.int32, "group_row_off")
    if out is None:
        out = (_empty((R, C // 2), torch.uint8, x), _empty((R, C // 16), torch.uint8, x),
               _empty((G,), torch.float32, x))
    codes, sf, ts = out
    rc = lib().nvfp4_quant_46_noalloc(_p(x), dt, R, C, _p(group_row_off), G, mode, pre_op, _p(codes), _p(sf),
                                      _p(ts), _stream())
    _check(rc, "nvfp4_quant_46_noalloc")
    return codes, sf, ts


def nvfp4_quant_requant_T(x, n_groups, seed=1, stream_id=0):
    """Weights [G*R_g, C] float32 -> NVFP4 mode 6 (codes, sf, ts per group) and
    its transposed MXFP8 SR copy (mx_codes [C*rows], mx_sf [C*rows/32]) in one pass."""
    _dev(x, torch.float32, "x")
    R, C = x.shape
    codes = _empty((R, C // 2), torch.uint8, x)
    sf = _empty((R, C // 16), torch.uint8, x)
    ts = _empty((n_groups,), torch.float32, x)
    mc = _empty((C * R,), torch.uint8, x)
    ms = _empty((C * R // 32,), torch.uint8, x)
    ws = _ws(lib().nvfp4_quant_requant_T_ws_bytes(n_groups), x)
    rc = lib().nvfp4_quant_requant_T(_p(x), R, C, n_groups, _p(codes), _p(sf), _p(ts), seed, stream_id, _p(mc),
                                     _p(ms), _p(ws), ws.numel(), _stream())
    _check(rc, "nvfp4_quant_requant_T")
    return codes, sf, ts, mc, ms


def mxfp8_quant_requant_T(x, n_groups, seed=1, stream_id=0):
    """Weights [G*R_g, C] float32 -> MXFP8 RNE row-wise (codes [R, C], sf [R, C/32])
    and its transposed MXFP8 SR copy (t_codes [C*R], t_sf [C*R/32]) in one pass."""
    _dev(x, torch.float32, "x")
    R, C = x.shape
    codes = _empty((R, C), torch.uint8, x)
    sf = _empty((R, C // 32), torch.uint8, x)
    tc = _empty((C * R,), torch.uint8, x)
    ts = _empty((C * R // 32,), torch.uint8, x)
    rc = lib().mxfp8_quant_requant_T(_p(x), R, C, n_groups, seed, stream_id, _p(codes), _p(sf), _p(tc), _p(ts),
                                     _stream())
    _check(rc, "mxfp8_quant_requant_T")
    return codes, sf, tc, ts


def nvfp4_dequant(codes, sf, ts, group_row_off=None, ts_per_group=False):
    R, H = codes.shape
    G = 1 if group_row_off is None else group_row_off.numel() - 1
    out = _empty((R, 2 * H), torch.float32, codes)
    rc = lib().nvfp4_dequant(_p(codes), _p(sf), _p(ts), int(ts_per_group), _p(group_row_off), G, R, 2 * H, _p(out),
                             _stream())
    _check(rc, "nvfp4_dequant")
    return out


# --------------------------------------------------------------------- MXFP8

def mxfp8_requant_sr_T(codes, sf, ts, group_row_off, group_off_pad, ts_per_group=True, seed=1, stream_id=0,
                       max_pr=None, sf_layout=SF_ROWS):
    """NVFP4 [R, C] -> MXFP8 SR, group-major padded: (codes [C*P], sf [C*P/32]) with P = max_pr;
    scales row-major per group (SF_ROWS) or block-major (SF_BLOCKS)."""
    R, H = codes.shape
    C = 2 * H
    G = group_row_off.numel() - 1
    _dev(group_row_off, torch.int32, "group_row_off")
    _dev(group_off_pad, torch.int32, "group_off_pad")
    if max_pr is None:
        max_pr = max_padded_rows(R, G)
    oc = _empty((C * max_pr,), torch.uint8, codes)
    os_ = _empty((C * max_pr // 32,), torch.uint8, codes)
    rc = lib().mxfp8_requant_sr_T(_p(codes), _p(sf), _p(ts), int(ts_per_group), R, C, _p(group_row_off),
                                  _p(group_off_pad), G, max_pr, seed, stream_id, int(sf_layout), _p(oc), _p(os_),
                                  _stream())
    _check(rc, "mxfp8_requant_sr_T")
    return oc, os_


def mxfp8_requant_mx_sr_T(codes, sf, group_row_off, group_off_pad, seed=1, stream_id=0, max_pr=None,
                          sf_layout=SF_ROWS):
    """MXFP8 row-wise [R, C] -> MXFP8 SR transposed, group-major padded: (codes [C*P], sf [C*P/32])."""
    R, C = codes.shape
    G = group_row_off.numel() - 1
    _dev(group_row_off, torch.int32, "group_row_off")
    _dev(group_off_pad, torch.int32, "group_off_pad")
    if max_pr is None:
        max_pr = max_padded_rows(R, G)
    oc = _empty((C * max_pr,), torch.uint8, codes)
    os_ = _empty((C * max_pr // 32,), torch.uint8, codes)
    rc = lib().mxfp8_requant_mx_sr_T(_p(codes), _p(sf), R, C, _p(group_row_off), _p(group_off_pad), G, max_pr, seed,
                                     stream_id, int(sf_layout), _p(oc), _p(os_), _stream())
    _check(rc, "mxfp8_requant_mx_sr_T")
    return oc, os_


def mxfp8_quant(x, rows=None, transpose=False, row_map=None, map_div=1, row_scale=None, dsilu_src=None,
                group_row_off=None, group_off_pad=None, max_pr=None, rnd=RNE, seed=0, stream_id=0,
                sf_layout=SF_ROWS, pre_op=PRE_NONE):
    """MXFP8 of a gradient (see moe4.h).  Row mode -> ([rows, C], [rows, C/32]);
    transposed -> (codes [C*max_pr], sf [C*max_pr/32]), scales per group
    row-major (SF_ROWS) or block-major (SF_BLOCKS)."""
    dt = {torch.bfloat16: BF16, torch.float32: F32}.get(x.dtype)
    if dt is None:
        raise ValueError("mxfp8_quant: x must be bf16 or float32")
    _dev(x, x.dtype, "x")
    C = x.shape[1]
    R = (row_map.numel() if row_map is not None else x.shape[0]) if rows is None else rows
    if row_map is not None:
        _dev(row_map, torch.int32, "row_map")
    if row_scale is not None:
        _dev(row_scale, torch.float32, "row_scale")
    if dsilu_src is not None:
        _dev(dsilu_src, torch.bfloat16, "dsilu_src")
    if transpose:
        G = group_row_off.numel() - 1
        if max_pr is None:
            max_pr = max_padded_rows(R, G)
        oc = _empty((C * max_pr,), torch.uint8, x)
        os_ = _empty((C * max_pr // 32,), torch.uint8, x)
    else:
        G = 0
        max_pr = 0
        oc = _empty((R, C), torch.uint8, x)
        os_ = _empty((R, C // 32), torch.uint8, x)
    mode = 0 if not transpose else (2 if sf_layout == SF_BLOCKS else 1)
    rc = lib().mxfp8_quant(_p(x), dt, R, C, _p(row_map), map_div, _p(row_scale), _p(dsilu_src), pre_op, mode,
                           _p(group_row_off), _p(group_off_pad), G, max_pr, rnd, seed, stream_id, _p(oc), _p(os_),
                           _stream())
    _check(rc, "mxfp8_quant")
    return oc, os_


def mxfp8_quant_rows_T(x, group_row_off, group_off_pad, rows=None, row_map=None, map_div=1, row_scale=None,
                       dsilu_src=None, max_pr=None, rnd=RNE, seed=0, stream_id=0, sf_layout=SF_ROWS):
    """Both MXFP8 copies of a gradient from one read (see moe4.h): returns
    (row_codes [rows, C], row_sf [rows, C/32], t_codes [C*max_pr], t_sf [C*max_pr/32])."""
    dt = {torch.bfloat16: BF16, torch.float32: F32}.get(x.dtype)
    if dt is None:
        raise ValueError("mxfp8_quant_rows_T: x must be bf16 or float32")
    _dev(x, x.dtype, "x")
    C = x.shape[1]
    R = (row_map.numel() if row_map is not None else x.shape[0]) if rows is None else rows
    if row_map is not None:
        _dev(row_map, torch.int32, "row_map")
    if row_scale is not None:
        _dev(row_scale, torch.float32, "row_scale")
    if dsilu_src is not None:
        _dev(dsilu_src, torch.bfloat16, "dsilu_src")
    _dev(group_row_off, torch.int32, "group_row_off")
    _dev(group_off_pad, torch.int32, "group_off_pad")
    G = group_row_off.numel() - 1
    if max_pr is None:
        max_pr = max_padded_rows(R, G)
    rc_ = _empty((R, C), torch.uint8, x)
    rs_ = _empty((R, C // 32), torch.uint8, x)
    tc = _empty((C * max_pr,), torch.uint8, x)
    ts = _empty((C * max_pr // 32,), torch.uint8, x)
    rc = lib().mxfp8_quant_rows_T(_p(x), dt, R, C, _p(row_map), map_div, _p(row_scale), _p(dsilu_src),
                                  _p(group_row_off), _p(group_off_pad), G, max_pr, rnd, seed, stream_id, sf_layout,
                                  _p(rc_), _p(rs_), _p(tc), _p(ts), _stream())
    _check(rc, "mxfp8_quant_rows_T")
    return rc_, rs_, tc, ts


def mxfp8_requant_mx4_sr_T(codes, sf, group_row_off, group_off_pad, seed=1, stream_id=0, max_pr=None,
                           sf_layout=SF_ROWS):
    """MXFP4 row-wise [R, C] -> MXFP8 SR transposed, group-major padded: (codes [C*P], sf [C*P/32])."""
    _arg(codes, torch.uint8, (None, None), "codes")
    R, C = codes.shape[0], 2 * codes.shape[1]
    _arg(sf, torch.uint8, (R, C // 32), "sf", codes)
    _arg(group_row_off, torch.int32, (None,), "group_row_off", codes)
    G = group_row_off.numel() - 1
    _arg(group_off_pad, torch.int32, (G + 1,), "group_off_pad", codes)
    if max_pr is None:
        max_pr = max_padded_rows(R, G)
    oc = _empty((C * max_pr,), torch.uint8, codes)
    os_ = _empty((C * max_pr // 32,), torch.uint8, codes)
    _run("mxfp8_requant_mx4_sr_T", codes, codes, sf, R, C, group_row_off, group_off_pad, G, max_pr,
         seed, stream_id, int(sf_layout), oc, os_)
    return oc, os_


# --------------------------------------------------------------------- MXFP4

def mxfp4_quant(x, pre_op=PRE_NONE, out_map=None, copies=1, out=None):
    """MXFP4 of x [R, C] (bf16 or float32) -> (codes [R, C/2] u8, sf [R, C/32] u8).
    out_map [R*copies] int32: row r goes to the output rows out_map[r*copies + j]
    (e.g. moe_route_topk's inv_perm, copies = k: the dispatch); the outputs then
    have R*copies rows; name each row once.  out: optional (codes, sf) tensors to
    write into; rows that out_map does not name keep what they hold."""
    dt = {torch.bfloat16: BF16, torch.float32: F32}.get(x.dtype)
    if dt is None:
        raise ValueError("mxfp4_quant: x must be bf16 or float32")
    _arg(x, x.dtype, (None, None), "x")
    R, C = x.shape
    if out_map is not None:
        _arg(out_map, torch.int32, (R * copies,), "out_map", x)
    elif copies != 1:
        raise ValueError("mxfp4_quant: copies needs out_map")
    if out is None:
        out = (_empty((R * copies, C // 2), torch.uint8, x), _empty((R * copies, C // 32), torch.uint8, x))
    codes, sf = out
    _arg(codes, torch.uint8, (None if out_map is not None else R, C // 2), "out codes", x)
    _arg(sf, torch.uint8, (codes.shape[0], C // 32), "out sf", x)
    _run("mxfp4_quant", x, x, dt, R, C, out_map, copies, codes.shape[0], int(pre_op), codes, sf)
    return codes, sf


def mxfp4_dequant(codes, sf, out_dtype=torch.float32):
    """The values of MXFP4 codes [R, C/2], scales [R, C/32]: [R, C] float32 or bf16 (both exact)."""
    dt = {torch.bfloat16: BF16, torch.float32: F32}.get(out_dtype)
    if dt is None:
        raise ValueError("mxfp4_dequant: out_dtype must be bf16 or float32")
    _arg(codes, torch.uint8, (None, None), "codes")
    R, C = codes.shape[0], 2 * codes.shape[1]
    _arg(sf, torch.uint8, (R, C // 32), "sf", codes)
    out = _empty((R, C), out_dtype, codes)
    _run("mxfp4_dequant", codes, codes, sf, R, C, out, dt)
    return out


# ------------------------------------------------------------------- routing

def moe_route_topk(logits, k, bias=None):
    """Top-k routing + stable permutation.  Returns dict(idx, gates, off, off_pad, perm, inv_perm)."""
    _dev(logits, torch.float32, "logits")
    T, E = logits.shape
    if bias is not None:
        _dev(bias, torch.float32, "bias")
    idx = _empty((T, k), torch.int32, logits)
    gates = _empty((T, k), torch.float32, logits)
    off = _empty((E + 1,), torch.int32, logits)
    off_pad = _empty((E + 1,), torch.int32, logits)
    perm = _empty((T * k,), torch.int32, logits)
    inv = _empty((T * k,), torch.int32, logits)
    ws = _ws(lib().moe_route_topk_ws_bytes(T, E, k), logits)
    rc = lib().moe_route_topk(_p(logits), _p(bias), T, E, k, _p(idx), _p(gates), _p(off), _p(off_pad), _p(perm),
                              _p(inv), _p(ws), ws.numel(), _stream())
    _check(rc, "moe_route_topk")
    return dict(idx=idx, gates=gates, off=off, off_pad=off_pad, perm=perm, inv_perm=inv)


def moe_gather_rows(codes, sf, perm, k):
    n_in, H = codes.shape
    A = perm.numel()
    oc = _empty((A, H), torch.uint8, codes)
    os_ = _empty((A, sf.shape[1]), torch.uint8, codes)
    rc = lib().moe_gather_rows(_p(codes), _p(sf), n_in, 2 * H, _p(perm), k, A, _p(oc), _p(os_), _stream())
    _check(rc, "moe_gather_rows")
    return oc, os_


# --------------------------------------------------------------------- GEMMs

def moe_grouped_gemm_fwd(a_codes, a_sf, a_ts, b_codes, b_sf, b_ts, expert_off, out_dtype=torch.bfloat16,
                         a_ts_per_group=False):
    """NVFP4 A [M, K] x NVFP4 B [E, N, K] grouped by expert_off -> C [M, N] (bf16 or float32)."""
    M, Kh = a_codes.shape
    E, N, _ = b_codes.shape
    c = _empty((M, N), out_dtype, a_codes)
    cd = BF16 if out_dtype == torch.bfloat16 else F32
    rc = lib().moe_grouped_gemm_fwd(_p(a_codes), _p(a_sf), _p(a_ts), int(a_ts_per_group), _p(b_codes), _p(b_sf),
                                    _p(b_ts), _p(expert_off), E, M, N, 2 * Kh, _p(c), cd, _stream())
    _check(rc, "moe_grouped_gemm_fwd")
    return c


def moe_grouped_gemm_fwd_silu_amax(a_codes, a_sf, a_ts, b_codes, b_sf, b_ts, expert_off, a_ts_per_group=False):
    """moe_grouped_gemm_fwd with bf16 U, plus each expert's max |silu(U)| as float bits
    in a workspace that nvfp4_quant_46(U, ..., PRE_SILU_AMAX, ws=...) takes.
    Raises Moe4Unsupported when the shape selects other kernels.  -> (U, ws)"""
    M, Kh = a_codes.shape
    E, N, _ = b_codes.shape
    c = _empty((M, N), torch.bfloat16, a_codes)
    ws = _ws(lib().nvfp4_quant_46_ws_bytes(E), a_codes)
    rc = lib().moe_grouped_gemm_fwd_silu_amax(_p(a_codes), _p(a_sf), _p(a_ts), int(a_ts_per_group), _p(b_codes),
                                              _p(b_sf), _p(b_ts), _p(expert_off), E, M, N, 2 * Kh, _p(c), _p(ws),
                                              _stream())
    _check(rc, "moe_grouped_gemm_fwd_silu_amax")
    return c, ws


def moe_grouped_gemm_fwd_hmx8(a_codes, a_sf, a_ts, b_codes, b_sf, b_ts, expert_off, a_ts_per_group=False):
    """moe_grouped_gemm_fwd with float32 C, plus C's combine-path payload written by the
    same epilogue.  Raises Moe4Unsupported when the shape selects other kernels.
    -> (C, codes int8 [M, N], scales uint8 [M, N/32])"""
    M, Kh = a_codes.shape
    E, N, _ = b_codes.shape
    c = _empty((M, N), torch.float32, a_codes)
    codes = _empty((M, N), torch.int8, a_codes)
    sf = _empty((M, N // 32), torch.uint8, a_codes)
    rc = lib().moe_grouped_gemm_fwd_hmx8(_p(a_codes), _p(a_sf), _p(a_ts), int(a_ts_per_group), _p(b_codes),
                                         _p(b_sf), _p(b_ts), _p(expert_off), E, M, N, 2 * Kh, _p(c), _p(codes),
                                         _p(sf), _stream())
    _check(rc, "moe_grouped_gemm_fwd_hmx8")
    return c, codes, sf


def moe_grouped_gemm_bwd_dgrad(a_codes, a_sf, b_codes, b_sf, expert_off):
    """MXFP8 A [M, K] x MXFP8 B [E, N, K] grouped by expert_off -> float32 C [M, N]."""
    M, K = a_codes.shape
    E = expert_off.numel() - 1
    N = b_codes.numel() // (E * K)
    c = _empty((M, N), torch.float32, a_codes)
    rc = lib().moe_grouped_gemm_bwd_dgrad(_p(a_codes), _p(a_sf), _p(b_codes), _p(b_sf), _p(expert_off), E, M, N, K,
                                          _p(c), _stream())
    _check(rc, "moe_grouped_gemm_bwd_dgrad")
    return c


def moe_grouped_gemm_mx(a_codes, a_sf, b_codes, b_sf, expert_off, out_dtype=torch.float32):
    """MXFP8 A [M, K] x MXFP8 B [E, N, K] per expert -> C [M, N] (float32 or bf16)."""
    M, K = a_codes.shape
    E = expert_off.numel() - 1
    N = b_codes.numel() // (E * K)
    cd = {torch.float32: F32, torch.bfloat16: BF16}[out_dtype]
    c = _empty((M, N), out_dtype, a_codes)
    rc = lib().moe_grouped_gemm_mx(_p(a_codes), _p(a_sf), _p(b_codes), _p(b_sf), _p(expert_off), E, M, N, K, _p(c),
                                   cd, _stream())
    _check(rc, "moe_grouped_gemm_mx")
    return c


WGRAD_SKIP_EMPTY = 1


def moe_grouped_gemm_bwd_wgrad(a_codes, a_sf, b_codes, b_sf, expert_off_pad, N1, N2, dw=None, beta=0.0,
                               skip_empty=False):
    """Group-major padded MXFP8 A [N1][P_e], B [N2][P_e] per expert -> dw [E, N1, N2] float32.
    skip_empty: experts without rows keep whatever dw holds (see moe4.h)."""
    E = expert_off_pad.numel() - 1
    if dw is None:
        dw = _empty((E, N1, N2), torch.float32, a_codes)
    rc = lib().moe_grouped_gemm_bwd_wgrad(_p(a_codes), _p(a_sf), _p(b_codes), _p(b_sf), _p(expert_off_pad), E, N1,
                                          N2, _p(dw), beta, WGRAD_SKIP_EMPTY if skip_empty else 0, _stream())
    _check(rc, "moe_grouped_gemm_bwd_wgrad")
    return dw


def moe_grouped_gemm_bwd(dy_codes, dy_sf, wT_codes, wT_sf, dyT_codes, dyT_sf, xT_codes, xT_sf, expert_off,
                         expert_off_pad, Nin, Nout, dw=None, beta=0.0, skip_empty=False):
    """dgrad and wgrad of one expert linear in one call: returns (dx float32
    [M, Nin], dw float32 [E, Nout, Nin]).  dy row-wise [M, Nout], W^T requantised
    [E][Nin][Nout], dy and x transposed group-major [Nout][P_e] / [Nin][P_e]
    with block-major scales."""
    M = dy_codes.shape[0]
    E = expert_off.numel() - 1
    dx = _empty((M, Nin), torch.float32, dy_codes)
    if dw is None:
        dw = _empty((E, Nout, Nin), torch.float32, dy_codes)
    rc = lib().moe_grouped_gemm_bwd(_p(dy_codes), _p(dy_sf), _p(wT_codes), _p(wT_sf), _p(dyT_codes), _p(dyT_sf),
                                    _p(xT_codes), _p(xT_sf), _p(expert_off), _p(expert_off_pad), E, M, Nin, Nout,
                                    _p(dx), _p(dw), beta, WGRAD_SKIP_EMPTY if skip_empty else 0, _stream())
    _check(rc, "moe_grouped_gemm_bwd")
    return dx, dw


def moe_grouped_gemm_mx4(a_codes, a_sf, b_codes, b_sf, expert_off, out_dtype=torch.bfloat16):
    """MXFP4 A [M, K] x MXFP4 B [E, N, K] grouped by expert_off -> C [M, N] (bf16 or float32)."""
    cd = {torch.float32: F32, torch.bfloat16: BF16}.get(out_dtype)
    if cd is None:
        raise ValueError("moe_grouped_gemm_mx4: out_dtype must be bf16 or float32")
    _arg(a_codes, torch.uint8, (None, None), "a_codes")
    M, Kh = a_codes.shape
    _arg(a_sf, torch.uint8, (M, Kh // 16), "a_sf", a_codes)
    _arg(b_codes, torch.uint8, (None, None, Kh), "b_codes", a_codes)
    E, N, _ = b_codes.shape
    _arg(b_sf, torch.uint8, (E, N, Kh // 16), "b_sf", a_codes)
    _arg(expert_off, torch.int32, (E + 1,), "expert_off", a_codes)
    c = _empty((M, N), out_dtype, a_codes)
    _run("moe_grouped_gemm_mx4", a_codes, a_codes, a_sf, b_codes, b_sf, expert_off, E, M, N,
         2 * Kh, c, cd)
    return c


# ------------------------------------------------------------------ BF16 GEMMs

def _bf16_rows(x, row_map, map_div, name):
    """The (gathered) bf16 operand's checks -> rows of the product."""
    _arg(x, torch.bfloat16, (None, None), name)
    if row_map is None:
        if map_div != 1:
            raise ValueError(f"{name}: map_div needs a map")
        return x.shape[0]
    _arg(row_map, torch.int32, (None,), f"{name}'s map", x)
    return row_map.numel()


def _row_scale(s, x, row_map, map_div, name):
    """Check a row scale of x: one per row, or with a map one per entry it may hold."""
    return s if s is None else _arg(s, torch.float32, (x.shape[0] * (1 if row_map is None else map_div),), name, x)


def _out_dtype(dtype, name):
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(dtype)
    if dt is None:
        raise ValueError(f"{name}: out_dtype must be bf16 or float32")
    return dt


def moe_grouped_gemm_bf16(a, w, expert_off, bias=None, act=ACT_NONE, residual=None, row_map=None, map_div=1,
                          out_dtype=torch.bfloat16, save_pre=False, out=None):
    """act(A . w[e]^T + bias[e]) + residual per expert -> (c [M, N], pre [M, N] bf16 or None).
    a [R, K] bf16, w [E, N, K] bf16, bias [E, N] float32, residual [M, N] of
    out_dtype; row_map [M] int32: row r of A is a[row_map[r] // map_div].  out: a
    tensor for c (it may be the residual)."""
    dt = _out_dtype(out_dtype, "moe_grouped_gemm_bf16")
    M = _bf16_rows(a, row_map, map_div, "a")
    K = a.shape[1]
    _arg(w, torch.bfloat16, (None, None, K), "w", a)
    E, N, _ = w.shape
    _arg(expert_off, torch.int32, (E + 1,), "expert_off", a)
    if bias is not None:
        _arg(bias, torch.float32, (E, N), "bias", a)
    if residual is not None:
        _arg(residual, out_dtype, (M, N), "residual", a)
    c = _empty((M, N), out_dtype, a) if out is None else _arg(out, out_dtype, (M, N), "out", a)
    pre = _empty((M, N), torch.bfloat16, a) if save_pre else None
    _run("moe_grouped_gemm_bf16", a, a, a.shape[0], row_map, map_div, w, bias, expert_off, E, M, N, K, int(act), residual,
         c, dt, pre)
    return c, pre


def moe_gated_gemm_bf16(a, w, expert_off, bias=None, act=ACT_SILU, row_map=None, map_div=1, save=True):
    """The gated block's first half: act(A . w[e, 0]^T + b) * (A . w[e, 1]^T + b') ->
    (h [M, F] bf16, gu [M, 2, F] bf16 or None: the two products, for the backward).
    a [R, K] bf16 (gathered as in moe_grouped_gemm_bf16), w [E, 2, F, K] bf16, bias [E, 2, F] float32."""
    M = _bf16_rows(a, row_map, map_div, "a")
    K = a.shape[1]
    _arg(w, torch.bfloat16, (None, 2, None, K), "w", a)
    E, _, F, _ = w.shape
    _arg(expert_off, torch.int32, (E + 1,), "expert_off", a)
    if bias is not None:
        _arg(bias, torch.float32, (E, 2, F), "bias", a)
    h = _empty((M, F), torch.bfloat16, a)
    gu = _empty((M, 2, F), torch.bfloat16, a) if save else None
    _run("moe_gated_gemm_bf16", a, a, a.shape[0], row_map, map_div, w, bias, expert_off, E, M, F, K, int(act), h, gu)
    return h, gu


def moe_grouped_gemm_bf16_dgrad(dy, w, expert_off, pre=None, act=ACT_NONE, row_scale=None, row_map=None, map_div=1,
                                out_dtype=torch.bfloat16, add=None, out=None):
    """Input gradient: z = row_scale * (dY . w[e]), with pre through the activation that made the
    input -> (dx [M, K], hs [M, K] bf16 or None): z + add, or z * act'(pre) + add and row_scale *
    act(pre).  add [M, K] of out_dtype; out: a tensor for dx (it may be add).
    dy [R, N] bf16 (gathered as above), w [E, N, K] bf16, pre [M, K] bf16, row_scale float32:
    [M] by row, or with a map [R * map_div] by the map's entry (the gates, flat)."""
    dt = _out_dtype(out_dtype, "moe_grouped_gemm_bf16_dgrad")
    M = _bf16_rows(dy, row_map, map_div, "dy")
    N = dy.shape[1]
    _arg(w, torch.bfloat16, (None, N, None), "w", dy)
    E, _, K = w.shape
    _arg(expert_off, torch.int32, (E + 1,), "expert_off", dy)
    _row_scale(row_scale, dy, row_map, map_div, "row_scale")
    if pre is not None:
        _arg(pre, torch.bfloat16, (M, K), "pre", dy)
    if add is not None:
        _arg(add, out_dtype, (M, K), "add", dy)
    dx = _empty((M, K), out_dtype, dy) if out is None else _arg(out, out_dtype, (M, K), "out", dy)
    hs = _empty((M, K), torch.bfloat16, dy) if pre is not None else None
    _run("moe_grouped_gemm_bf16_dgrad", dy, dy, dy.shape[0], row_map, map_div, row_scale, w, expert_off, E, M, N, K, int(act),
         pre, add, dx, dt, hs)
    return dx, hs


def moe_gated_gemm_bf16_dgrad(dy, w, gu, expert_off, act=ACT_SILU, row_scale=None, row_map=None, map_div=1):
    """Through the output projection and the gated block: dh = row_scale * (dY . w[e]) ->
    (dgu [M, 2, F] bf16: dh u act'(g) and dh act(g), hs [M, F] bf16 = row_scale * act(g) * u).
    dy [R, N] bf16 (gathered as above), w [E, N, F] bf16, gu [M, 2, F] bf16 as the forward kept it."""
    M = _bf16_rows(dy, row_map, map_div, "dy")
    N = dy.shape[1]
    _arg(w, torch.bfloat16, (None, N, None), "w", dy)
    E, _, F = w.shape
    _arg(expert_off, torch.int32, (E + 1,), "expert_off", dy)
    _arg(gu, torch.bfloat16, (M, 2, F), "gu", dy)
    _row_scale(row_scale, dy, row_map, map_div, "row_scale")
    dgu = _empty((M, 2, F), torch.bfloat16, dy)
    hs = _empty((M, F), torch.bfloat16, dy)
    _run("moe_gated_gemm_bf16_dgrad", dy, dy, dy.shape[0], row_map, map_div, row_scale, w, expert_off, E, M, N, F, int(act), gu,
         dgu, hs)
    return dgu, hs


def moe_grouped_gemm_bf16_wgrad(dy, a, expert_off, dy_map=None, a_map=None, map_div=1, dw=None, beta=0.0, skip_empty=False,
                                bias_grad=False, db_scale=None, db=None):
    """dw[e] = beta dw[e] + sum over e's rows of dY^T . A -> (dw [E, N, K] float32, db [E, N]
    float32 or None: beta db[e] + sum of db_scale * dY).  dy [R, N], a [R', K] bf16, each
    gathered if its map is given; skip_empty as in moe_grouped_gemm_bwd_wgrad."""
    if map_div != 1 and dy_map is None and a_map is None:
        raise ValueError("moe_grouped_gemm_bf16_wgrad: map_div needs a map")
    M = _bf16_rows(dy, dy_map, 1, "dy")
    _arg(a, torch.bfloat16, (M if a_map is None else None, None), "a", dy)
    if a_map is not None:
        _arg(a_map, torch.int32, (M,), "a's map", dy)
    N, K = dy.shape[1], a.shape[1]
    _arg(expert_off, torch.int32, (None,), "expert_off", dy)
    E = expert_off.numel() - 1
    if beta and (dw is None or (bias_grad and db is None)):
        raise ValueError("moe_grouped_gemm_bf16_wgrad: beta needs dw (and db) to add to")
    dw = _empty((max(E, 0), N, K), torch.float32, dy) if dw is None else _arg(dw, torch.float32, (E, N, K), "dw", dy)
    if db is not None:
        _arg(db, torch.float32, (E, N), "db", dy)
    elif bias_grad:
        db = _empty((max(E, 0), N), torch.float32, dy)
    _row_scale(db_scale, dy, dy_map, map_div, "db_scale")
    ws = _ws(lib().moe_grouped_gemm_bf16_wgrad_ws_bytes(E, M, N, K), dy)
    _run("moe_grouped_gemm_bf16_wgrad", dy, dy, dy.shape[0], dy_map, a, a.shape[0], a_map, map_div, expert_off, E, M, N, K, dw,
         float(beta), WGRAD_SKIP_EMPTY if skip_empty else 0, db_scale, db, ws, ws.numel())
    return dw, db


# ----------------------------------------------------------- combine / misc

def moe_combine_dropout(yp, gates, inv_perm, p, seed=1, stream_id=0, residual=None, out=None):
    """y [T, d] bf16 = residual + dropout(sum_j gates[t, j] * yp[inv_perm[t*k+j]]): an element is kept
    with probability 1 - p (to 2**-17) by the counter hash of (seed, stream_id, its index) and then
    scaled by the inverse.  residual [T, d] bf16; out: a tensor for y (it may be the residual)."""
    _arg(gates, torch.float32, (None, None), "gates")
    T, k = gates.shape
    _arg(yp, torch.float32, (T * k, None), "yp", gates)
    d = yp.shape[1]
    _arg(inv_perm, torch.int32, (T * k,), "inv_perm", gates)
    if residual is not None:
        _arg(residual, torch.bfloat16, (T, d), "residual", gates)
    y = _empty((T, d), torch.bfloat16, gates) if out is None else _arg(out, torch.bfloat16, (T, d), "out", gates)
    _run("moe_combine_dropout", gates, yp, gates, inv_perm, T, k, d, float(p), seed, stream_id, residual, y)
    return y


def moe_dropout_backward(dy, p, seed=1, stream_id=0, out=None):
    """The gradient of moe_combine_dropout in the combined sum (the same p, seed and stream_id):
    dy [T, d] bf16 where kept, scaled, else 0.  out: a tensor for it (it may be dy)."""
    _arg(dy, torch.bfloat16, (None, None), "dy")
    T, d = dy.shape
    dx = _empty((T, d), torch.bfloat16, dy) if out is None else _arg(out, torch.bfloat16, (T, d), "out", dy)
    _run("moe_dropout_backward", dy, dy, T, d, float(p), seed, stream_id, dx)
    return dx


def moe_combine(yp, gates, inv_perm):
    T, k = gates.shape
    d = yp.shape[1]
    y = _empty((T, d), torch.bfloat16, yp)
    rc = lib().moe_combine(_p(yp), _p(gates), _p(inv_perm), T, k, d, _p(y), _stream())
    _check(rc, "moe_combine")
    return y


def moe_hmx8_quant(x):
    """Combine-path payload of x [rows, cols] float32: (codes int8, scales uint8 [rows, cols/32])."""
    _dev(x, torch.float32, "moe_hmx8_quant")
    rows, cols = x.shape
    codes = _empty((rows, cols), torch.int8, x)
    sf = _empty((rows, cols // 32), torch.uint8, x)
    rc = lib().moe_hmx8_quant(_p(x), rows, cols, _p(codes), _p(sf), _stream())
    _check(rc, "moe_hmx8_quant")
    return codes, sf


def moe_hmx8_dequant(codes, sf):
    rows, cols = codes.shape
    out = _empty((rows, cols), torch.float32, codes)
    rc = lib().moe_hmx8_dequant(_p(codes), _p(sf), rows, cols, _p(out), _stream())
    _check(rc, "moe_hmx8_dequant")
    return out


def moe_combine_hmx8(codes, sf, gates, inv_perm):
    T, k = gates.shape
    d = codes.shape[1]
    y = _empty((T, d), torch.bfloat16, codes)
    rc = lib().moe_combine_hmx8(_p(codes), _p(sf), _p(gates), _p(inv_perm), T, k, d, _p(y), _stream())
    _check(rc, "moe_combine_hmx8")
    return y


def moe_unpermute_sum(dxp, inv_perm, T, k):
    d = dxp.shape[1]
    dx = _empty((T, d), torch.bfloat16, dxp)
    rc = lib().moe_unpermute_sum(_p(dxp), _p(inv_perm), T, k, d, _p(dx), _stream())
    _check(rc, "moe_unpermute_sum")
    return dx


def moe_dgates(dy, yp, inv_perm, k):
    """Gate gradient dg [T, k] float32: dg[t, j] = <dy[t], yp[inv_perm[t*k + j]]>."""
    _dev(dy, torch.bfloat16, "dy")
    _dev(yp, torch.float32, "yp")
    _dev(inv_perm, torch.int32, "inv_perm")
    T, d = dy.shape
    dg = _empty((T, k), torch.float32, dy)
    rc = lib().moe_dgates(_p(dy), _p(yp), _p(inv_perm), T, k, d, _p(dg), _stream())
    _check(rc, "moe_dgates")
    return dg


def moe_route_backward(dg, gates, topk_idx, E):
    """dlogits [T, E] float32: softmax backward over each token's selected experts."""
    _dev(dg, torch.float32, "dg")
    _dev(gates, torch.float32, "gates")
    _dev(topk_idx, torch.int32, "topk_idx")
    T, k = gates.shape
    out = _empty((T, E), torch.float32, gates)
    rc = lib().moe_route_backward(_p(dg), _p(gates), _p(topk_idx), T, E, k, _p(out), _stream())
    _check(rc, "moe_route_backward")
    return out


# -------------------------------------------------------------------- router

def moe_router_logits(x, w):
    """BF16 router GEMM: x [T, d] bf16, w [E, d] bf16 -> logits [T, E] float32."""
    _dev(x, torch.bfloat16, "x")
    _dev(w, torch.bfloat16, "w")
    T, d = x.shape
    E = w.shape[0]
    out = _empty((T, E), torch.float32, x)
    rc = lib().moe_router_logits(_p(x), _p(w), T, E, d, _p(out), _stream())
    _check(rc, "moe_router_logits")
    return out


def moe_unpermute_sum_router(dxp, inv_perm, T, k, dlogits, topk_idx, w):
    """dx [T, d] bf16: the un-permuting sum of dxp plus the router's input
    gradient sum_j dlogits[t, e_j] * w[e_j] (see moe4.h for the order)."""
    _dev(dxp, torch.float32, "dxp")
    _dev(dlogits, torch.float32, "dlogits")
    _dev(topk_idx, torch.int32, "topk_idx")
    _dev(w, torch.bfloat16, "w")
    d = dxp.shape[1]
    E = w.shape[0]
    dx = _empty((T, d), torch.bfloat16, dxp)
    rc = lib().moe_unpermute_sum_router(_p(dxp), _p(inv_perm), T, k, d, _p(dlogits), _p(topk_idx), E, _p(w), _p(dx),
                                        _stream())
    _check(rc, "moe_unpermute_sum_router")
    return dx


def moe_router_wgrad(x, dlogits, perm, expert_off, k):
    """dW_r [E, d] float32 = sum over the tokens routed to e of dlogits[t, e] * x[t]."""
    _dev(x, torch.bfloat16, "x")
    _dev(dlogits, torch.float32, "dlogits")
    T, d = x.shape
    E = dlogits.shape[1]
    dw = _empty((E, d), torch.float32, x)
    ws = _ws(lib().moe_router_wgrad_ws_bytes(T, E, k, d), x)
    rc = lib().moe_router_wgrad(_p(x), _p(dlogits), _p(perm), _p(expert_off), T, E, k, d, _p(dw), _p(ws), ws.numel(),
                                _stream())
    _check(rc, "moe_router_wgrad")
    return dw


def _mask_u8(mask, T, like):
    if mask is None:
        return None
    if mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    return _arg(mask, torch.uint8, (T,), "token_mask", like)


def moe_balance_loss(logits, topk_idx, bias=None, token_mask=None, seg_off=None):
    """Balance loss of the router per token segment (see moe4.h) -> dict(loss [S]
    float32, counts [S, E] int32, tokens [S] int32, probs [S, E] float32).
    token_mask [T] bool or uint8: False for padding; seg_off [S + 1] int32 token
    offsets (None: one segment)."""
    _arg(logits, torch.float32, (None, None), "logits")
    T, E = logits.shape
    _arg(topk_idx, torch.int32, (T, None), "topk_idx", logits)
    k = topk_idx.shape[1]
    if bias is not None:
        _arg(bias, torch.float32, (E,), "bias", logits)
    mask = _mask_u8(token_mask, T, logits)
    S = 1
    if seg_off is not None:
        _arg(seg_off, torch.int32, (None,), "seg_off", logits)
        S = seg_off.numel() - 1
    r = dict(loss=_empty((max(S, 0),), torch.float32, logits), counts=_empty((max(S, 0), E), torch.int32, logits),
             tokens=_empty((max(S, 0),), torch.int32, logits), probs=_empty((max(S, 0), E), torch.float32, logits))
    ws = _ws(lib().moe_balance_loss_ws_bytes(T, E, S), logits)
    _run("moe_balance_loss", logits, logits, bias, topk_idx, mask, seg_off, S, T, E, k,
         r["loss"], r["counts"], r["tokens"], r["probs"], ws, ws.numel())
    return r


def moe_balance_loss_backward(dloss, logits, counts, tokens, k, bias=None, token_mask=None, seg_off=None,
                              dlogits=None, out=None):
    """dlogits [T, E] float32 of sum_s dloss[s] * loss[s] (counts and tokens as
    moe_balance_loss returned them), added to ``dlogits`` if given; ``out`` (which
    may be ``dlogits``) receives it, else a new tensor."""
    _arg(logits, torch.float32, (None, None), "logits")
    T, E = logits.shape
    _arg(counts, torch.int32, (None, E), "counts", logits)
    S = counts.shape[0]
    _arg(dloss, torch.float32, (S,), "dloss", logits)
    _arg(tokens, torch.int32, (S,), "tokens", logits)
    if bias is not None:
        _arg(bias, torch.float32, (E,), "bias", logits)
    mask = _mask_u8(token_mask, T, logits)
    if seg_off is not None:
        _arg(seg_off, torch.int32, (S + 1,), "seg_off", logits)
    if dlogits is not None:
        _arg(dlogits, torch.float32, (T, E), "dlogits", logits)
    out = _empty((T, E), torch.float32, logits) if out is None else _arg(out, torch.float32, (T, E), "out", logits)
    _run("moe_balance_loss_backward", logits, dloss, logits, bias, counts, tokens, mask,
         seg_off, S, T, E, k, dlogits, out)
    return out


def moe_unpermute_sum_router_dense(dxp, inv_perm, T, k, dlogits, w):
    """dx [T, d] bf16: the un-permuting sum of dxp plus dlogits . w over all experts."""
    _arg(dxp, torch.float32, (T * k, None), "dxp")
    d = dxp.shape[1]
    _arg(w, torch.bfloat16, (None, d), "w", dxp)
    E = w.shape[0]
    _arg(dlogits, torch.float32, (T, E), "dlogits", dxp)
    _arg(inv_perm, torch.int32, (T * k,), "inv_perm", dxp)
    dx = _empty((T, d), torch.bfloat16, dxp)
    _run("moe_unpermute_sum_router_dense", dxp, dxp, inv_perm, T, k, d, dlogits, E, w, dx)
    return dx


def moe_router_wgrad_dense(x, dlogits):
    """dW_r [E, d] float32 = dlogits^T . x over all tokens and experts."""
    _arg(x, torch.bfloat16, (None, None), "x")
    T, d = x.shape
    _arg(dlogits, torch.float32, (T, None), "dlogits", x)
    E = dlogits.shape[1]
    dw = _empty((E, d), torch.float32, x)
    ws = _ws(lib().moe_router_wgrad_dense_ws_bytes(T, E, d), x)
    _run("moe_router_wgrad_dense", x, x, dlogits, T, E, d, dw, ws, ws.numel())
    return dw


def moe4_debug_check():
    """Synchronise the current stream; raise Moe4Error on a failed launch and
    Moe4DeviceError on a device-side error report (which this clears)."""
    _check(lib().moe4_debug_check(_stream()), "moe4_debug_check")


def moe4_debug_force_wait_timeout(on):
    """Test hook: make nvfp4_quant_requant_T's bounded waits give up (see moe4.h)."""
    _check(lib().moe4_debug_force_wait_timeout(int(bool(on))), "moe4_debug_force_wait_timeout")


def moe_silu_eval(u):
    _dev(u, torch.bfloat16, "u")
    s = _empty(u.shape, torch.float32, u)
    d = _empty(u.shape, torch.float32, u)
    rc = lib().moe_silu_eval(_p(u), u.numel(), _p(s), _p(d), _stream())
    _check(rc, "moe_silu_eval")
    return s, d
