"""Pins of the MXFP4 oracle: the scale rule and the codes against brute force
over all scales and codes, closed forms, and the exact decode."""
import numpy as np
import pytest

from oracle import formats as fmt
from oracle import mxfp4
from oracle import mxfp8 as mx
from oracle import nvfp4 as nv


def test_scale_exponent_is_the_least_that_does_not_saturate():
    rng = np.random.default_rng(0)
    a = np.concatenate([np.exp2(rng.uniform(-140, 127, 2000)), [6.0, 6.0 + 2 ** -20, 6.0 - 2 ** -20, 1.5, 3.0, 2.0 ** -149, 12.0]])
    a = a.astype(np.float32).astype(np.float64)
    e = mxfp4.scale_exponent(a)
    assert (a <= 6.0 * np.exp2(e.astype(float))).all()
    low = e > -127
    assert (a[low] > 6.0 * np.exp2(e[low] - 1.0)).all()
    assert mxfp4.scale_exponent([0.0])[0] == -127
    assert mxfp4.scale_exponent([float(np.finfo(np.float32).max)])[0] == 126


def test_codes_against_brute_force():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 96)) * np.exp2(rng.integers(-30, 30, (40, 1)))).astype(np.float32)
    codes, sf = mxfp4.quantize(x)
    q = nv.unpack_codes(codes)
    s = np.repeat(np.exp2(sf.astype(float) - 127), 32, axis=1)
    err = np.abs(x.astype(float) - mxfp4.dequant(codes, sf))
    grid = fmt.E2M1_MAG
    best = np.min(np.abs(np.abs(x.astype(float))[:, :, None] - grid * s[:, :, None]), axis=2)
    assert np.array_equal(err, best)                     # the nearest value, always
    assert np.array_equal((q >> 3) == 1, np.signbit(x))


def test_ties_go_to_the_even_code():
    x = np.zeros((1, 32), np.float32)
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25]     # e = 0
    codes, sf = mxfp4.quantize(x)
    assert sf[0, 0] == 127
    assert nv.unpack_codes(codes)[0, :9].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8]


def test_bits_per_value():
    codes, sf = mxfp4.quantize(np.ones((4, 64), np.float32))
    assert (codes.nbytes + sf.nbytes) * 8 / (4 * 64) == 4.25


def test_special_blocks():
    x = np.ones((1, 160), np.float32)
    x[0, 0], x[0, 40], x[0, 64:96], x[0, 96:128] = np.inf, np.nan, 0.0, -0.0
    codes, sf = mxfp4.quantize(x)
    assert sf[0].tolist() == [255, 255, 0, 0, 125]        # 1 = 4 * 2**-2
    v = mxfp4.dequant(codes, sf)
    assert np.isnan(v[0, :64]).all() and not v[0, 64:128].any() and (v[0, 128:] == 1).all()
    assert np.signbit(v[0, 96:128]).all()


@pytest.mark.parametrize("layout", [mx.SF_ROWS, mx.SF_BLOCKS])
def test_requant_equals_quantise_of_the_values(layout):
    """Grid values of one power of two per column stay themselves: SR leaves
    what E4M3 holds exactly unchanged."""
    x = np.tile(np.float32([1, 2, 3, 4]), (37, 16)).astype(np.float32)
    codes, sf = mxfp4.quantize(x)
    off = [0, 5, 5, 37]
    c, s = mxfp4.requant_sr_t(codes, sf, off, 1, 3, layout)
    for (a, b), blk in zip(zip(off[:-1], off[1:]), mx.dequant_transposed(c, s, off, 64, layout)):
        assert np.array_equal(blk[:, :b - a], x[a:b].T.astype(float))
        assert not blk[:, b - a:].any()


@pytest.mark.parametrize("layout", [mx.SF_ROWS, mx.SF_BLOCKS])
def test_requant_equals_the_float32_requantisation(layout):
    """Within float32's range the values are float32, and the transposed quantiser of those gives the same bytes."""
    rng = np.random.default_rng(6)
    codes, sf = mxfp4.quantize((rng.standard_normal((70, 96)) * np.exp2(rng.integers(-20, 20, (70, 1)))).astype(np.float32))
    off = [0, 1, 1, 40, 70]
    want = mx.quantize_transposed(mxfp4.dequant(codes, sf).astype(np.float32), off, mx.SR, 9, 18, layout)
    for a, b in zip(mxfp4.requant_sr_t(codes, sf, off, 9, 18, layout), want):
        assert np.array_equal(a, b)
