"""MXFP4 quantisation and its transposed requantisation to MXFP8 (test infrastructure).

MXFP4 is taken as E2M1 elements with one E8M0 scale per 32 values of a row
(the format of the 4-bit matrix hardware of the fourweekmba.com page's table,
with the power-of-two scales that gfx950's block-scaled products apply).

Block of 32 values v_i:
* scale exponent e: amax = max|v_i|; e = -127 if amax == 0, otherwise the least
  integer with amax <= 6 * 2**e, clamped to [-127, 127]; stored byte e + 127.
* code = E2M1(v_i * 2**-e), round to nearest, ties to even, signs kept.
* a block with an infinity or a NaN: scale byte 255, zero codes.

The transposed requantisation reads the exact values q * 2**e and follows
mxfp8.quantize_transposed with stochastic rounding; a source scale byte 255
gives the column blocks that meet it the scale byte 255.
"""
import numpy as np

from . import formats as fmt
from . import mxfp8 as mx
from . import nvfp4 as nv
from . import srhash

BLOCK = 32


def scale_exponent(amax):
    """Least integer e with amax <= 6 * 2**e, in [-127, 127] (-127 for 0); amax float64, finite."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.full(amax.shape, -127, dtype=np.int64)
    nz = amax > 0
    mant, ex = np.frexp(amax[nz])               # amax = mant * 2**ex = (mant * 2) * 2**(ex - 1)
    e[nz] = np.where(mant <= 0.75, ex - 3, ex - 2)
    return np.clip(e, -127, 127)


def quantize(x32):
    """x [R, C] float32 -> (packed codes [R, C/2] u8, scale bytes [R, C/32] u8)."""
    x = np.asarray(x32, dtype=np.float32)
    R, C = x.shape
    b = x.reshape(R, C // BLOCK, BLOCK).astype(np.float64)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    e = scale_exponent(np.max(np.abs(b), axis=2))
    q = fmt.e2m1_round(b * np.exp2(-e.astype(np.float64))[:, :, None])
    sf = np.where(bad, 255, e + 127).astype(np.uint8)
    return nv.pack_codes(np.asarray(q, dtype=np.uint8).reshape(R, C)), sf


def dequant(codes, sf):
    """Exact float64 values [R, C] (NaN under the scale byte 255)."""
    q = nv.unpack_codes(codes)
    s = np.asarray(sf, dtype=np.float64)
    s = np.where(np.asarray(sf) == 255, np.nan, np.exp2(s - 127.0))
    return fmt.e2m1_decode(q) * np.repeat(s, BLOCK, axis=1)


def requant_sr_t(codes, sf, group_row_off=None, seed=1, stream_id=0, sf_layout=mx.SF_ROWS):
    """MXFP4 [R, C] -> exact values (float64: 6 * 2**127 is past float32) ->
    transpose -> MXFP8 SR, in the layout of mxfp8.quantize_transposed (finite
    scale bytes)."""
    v = dequant(codes, sf)
    R, C = v.shape
    off = [0, R] if group_row_off is None else [int(o) for o in group_row_off]
    out_c, out_s = [], []
    for r0, r1 in zip(off[:-1], off[1:]):
        P = mx.pad32(r1 - r0)
        if P == 0:
            continue
        blk = np.zeros((C, P))
        blk[:, :r1 - r0] = v[r0:r1].T
        e = mx.mx_scale_exponent(np.abs(blk).reshape(C, P // 32, 32).max(axis=2))
        index = (r0 + np.arange(P, dtype=np.uint64))[None, :] * np.uint64(C) + np.arange(C, dtype=np.uint64)[:, None]
        w = blk * np.repeat(np.exp2(-e.astype(np.float64)), 32, axis=1)
        out_c.append(mx.round_sr(w, srhash.random16(seed, stream_id, index)).astype(np.uint8).reshape(-1))
        s = (e + 127).astype(np.uint8)
        out_s.append((s if sf_layout == mx.SF_ROWS else s.T).reshape(-1))
    return (np.concatenate(out_c), np.concatenate(out_s)) if out_c else (np.zeros(0, np.uint8), np.zeros(0, np.uint8))
