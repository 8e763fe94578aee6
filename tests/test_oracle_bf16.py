"""Pins of the BF16 layer's oracle: activations against closed forms and differences, products
against loops, the dropout mask against its rate and its invariants."""
import math

import numpy as np
import pytest

from oracle import bf16 as ob
from oracle import srhash


@pytest.mark.parametrize("x", [-30.0, -2.5, -0.1, 0.0, 0.3, 1.0, 4.0, 30.0])
def test_activations_closed_forms(x):
    assert math.isclose(float(ob.act(ob.SILU, x)[0]), x / (1 + math.exp(-x)), rel_tol=1e-14, abs_tol=1e-300)
    want = 0.5 * x * (1 + math.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    assert math.isclose(float(ob.act(ob.GELU, x)[0]), want, rel_tol=1e-12, abs_tol=1e-15)
    assert float(ob.act(ob.NONE, x)[0]) == x and float(ob.act(ob.NONE, x)[1]) == 1.0


@pytest.mark.parametrize("kind", [ob.SILU, ob.GELU])
def test_derivatives_against_differences(kind):
    x = np.linspace(-8, 8, 401)
    h = 1e-5
    num = (ob.act(kind, x + h)[0] - ob.act(kind, x - h)[0]) / (2 * h)
    assert np.abs(ob.act(kind, x)[1] - num).max() < 1e-9
    assert np.abs(ob.act(kind, x)[1]).max() < 1.13


@pytest.mark.parametrize("kind", [ob.SILU, ob.GELU])
def test_activation_limits(kind):
    f, d = ob.act(kind, np.array([-np.inf, np.inf, -1e30, 1e30, np.nan]))
    assert f[0] == 0 and np.signbit(f[0]) and f[1] == np.inf and f[2] == 0 and f[3] == 1e30 and np.isnan(f[4])
    assert list(d[:4]) == [0, 1, 0, 1] and np.isnan(d[4])


def test_products_against_loops():
    rng = np.random.default_rng(1)
    off = [1, 3, 3, 6]
    a, w, x = rng.standard_normal((7, 4)), rng.standard_normal((3, 5, 4)), rng.standard_normal((7, 5))
    z, m = ob.product(a, w, off, True)
    y, _ = ob.product(x, w, off, False)
    dw, _ = ob.wgrad(x, a, off)
    want = np.zeros((3, 5, 4))
    for r in range(7):
        e = 0 if 1 <= r < 3 else 2 if 3 <= r < 6 else None
        if e is None:
            assert np.isnan(z[r]).all() and np.isnan(y[r]).all()
            continue
        for n in range(5):
            assert math.isclose(z[r, n], sum(a[r, k] * w[e, n, k] for k in range(4)), rel_tol=1e-12)
            assert math.isclose(m[r, n], sum(abs(a[r, k] * w[e, n, k]) for k in range(4)), rel_tol=1e-12)
            for k in range(4):
                want[e, n, k] += x[r, n] * a[r, k]
        for k in range(4):
            assert math.isclose(y[r, k], sum(x[r, n] * w[e, n, k] for n in range(5)), rel_tol=1e-12)
    assert np.allclose(dw, want, rtol=1e-12) and (dw[1] == 0).all()


def test_gathered_rows():
    x = np.arange(6.0)[:, None]
    assert ob.rows(x, [7, 0, 11], 2)[:, 0].tolist() == [3, 0, 5]


def test_dropout_mask():
    T, d = 256, 1024
    for p in (0.1, 0.5, 0.9):
        keep, f = ob.keep_mask(T, d, p, 5, 4)
        q = round((1 - p) * 65536) / 65536
        # the mean of n = 2^18 draws: five standard deviations
        assert abs(keep.mean() - q) < 5 * math.sqrt(q * (1 - q) / (T * d)) and f == 1 / q
    assert ob.keep_mask(T, d, 0.0, 5, 4)[0].all() and not ob.keep_mask(T, d, 1.0, 5, 4)[0].any()
    a, b, c = (ob.keep_mask(T, d, 0.5, *k)[0] for k in ((5, 4), (6, 4), (5, 5)))
    for o in (b, c):                                  # another seed or stream: independent
        assert abs((a == o).mean() - 0.5) < 5 * 0.5 / math.sqrt(T * d)
    # a larger p drops all that a smaller one drops
    k1, k2 = ob.keep_mask(T, d, 0.2, 5, 4)[0], ob.keep_mask(T, d, 0.7, 5, 4)[0]
    assert not (k2 & ~k1).any()
    assert ob.keep_mask(1, 8, 0.5, 5, 4)[0][0].tolist() == (srhash.random16(5, 4, np.arange(8)) < 32768).tolist()


def test_combine_dropout_expectation_and_residual():
    rng = np.random.default_rng(2)
    yp, gates, inv, res = rng.standard_normal((8, 16)), rng.random((4, 2)), rng.permutation(8), rng.standard_normal((4, 16))
    full = ob.combine_dropout(yp, gates, inv, 0.0, 1, 0)
    assert np.allclose(full[1], gates[1, 0] * yp[inv[2]] + gates[1, 1] * yp[inv[3]])
    mean = np.mean([ob.combine_dropout(yp, gates, inv, 0.5, s, 0) for s in range(4000)], axis=0)
    # a kept value is doubled: the mean of n draws has the standard deviation |v| / sqrt(n)
    assert (np.abs(mean - full) < 5 * np.abs(full) / math.sqrt(4000) + 1e-12).all()
    assert np.array_equal(ob.combine_dropout(yp, gates, inv, 1.0, 1, 0, res), res)
