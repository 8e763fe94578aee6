"""Pins of the balance-loss oracle: closed forms, brute force, central differences."""
import numpy as np
import pytest

from oracle import balance
from oracle import route
from oracle import router


def test_even_router_has_loss_one_and_no_gradient():
    T, E, k = 12, 6, 2
    idx = np.stack([(2 * np.arange(T)) % E, (2 * np.arange(T) + 1) % E], 1)
    r = balance.balance_loss(np.zeros((T, E), np.float32), idx)
    assert np.isclose(r["loss"][0], 1.0, rtol=1e-14) and (r["counts"] == T * k // E).all() and r["tokens"][0] == T
    g = balance.balance_grad([1.0], np.zeros((T, E), np.float32), r["counts"], r["tokens"], k)
    assert np.abs(g).max() < 1e-16


def test_collapsed_router_has_loss_e_over_k():
    T, E, k = 5, 8, 2
    z = np.full((T, E), -np.inf, np.float32)
    z[:, 3] = z[:, 5] = 1.0
    r = balance.balance_loss(z, np.tile([3, 5], (T, 1)))
    assert np.isclose(r["loss"][0], E / k, rtol=1e-14)


def test_segments_and_mask_against_loops():
    rng = np.random.default_rng(2)
    T, E, k = 40, 7, 3
    z, bias = rng.standard_normal((T, E)).astype(np.float32), rng.standard_normal(E).astype(np.float32)
    mask = rng.random(T) < 0.7
    off = [0, 3, 3, 4, 30, 38]                       # tokens 38, 39 outside
    idx, _ = route.topk_gates(z, k, bias)
    r = balance.balance_loss(z, idx, bias, mask, off)
    for s in range(5):
        n, c, m = 0, np.zeros(E), np.zeros(E)
        for t in range(off[s], off[s + 1]):
            if mask[t]:
                n += 1
                v = np.exp((z[t] + bias).astype(np.float64))
                m += v / v.sum()
                for e in idx[t]:
                    c[e] += 1
        assert r["tokens"][s] == n and np.array_equal(r["counts"][s], c)
        want = E / (k * n) * (c * m / n).sum() if n else 0.0
        assert np.isclose(r["loss"][s], want, rtol=1e-12)


def test_gradient_against_differences():
    rng = np.random.default_rng(3)
    T, E, k = 9, 5, 2
    z = rng.standard_normal((T, E)).astype(np.float32)
    idx, _ = route.topk_gates(z, k)
    off, mask, w = [0, 4, 9], np.array([1, 1, 0, 1, 1, 1, 1, 0, 1], bool), np.array([0.7, -1.3])
    r = balance.balance_loss(z, idx, None, mask, off)
    g = balance.balance_grad(w, z, r["counts"], r["tokens"], k, None, mask, off)
    h = 2.0 ** -8
    for t in range(T):
        for e in range(E):
            d = []
            for sgn in (1, -1):
                y = z.copy()
                y[t, e] += np.float32(sgn * h)
                d.append((balance.balance_loss(y, idx, None, mask, off)["loss"] * w).sum())
            # step error O(h^2) of a loss with third derivatives of order one
            assert abs((d[0] - d[1]) / (2 * h) - g[t, e]) < 4 * h * h * np.abs(w).max()


def test_row_of_minus_infinities():
    z = np.zeros((2, 4), np.float32)
    z[1] = -np.inf
    r = balance.balance_loss(z, np.array([[0, 1], [0, 1]]))
    assert np.array_equal(r["probs"][0], [0.125] * 4)
    assert not balance.balance_grad([1.0], z, r["counts"], r["tokens"], 2)[1].any()


@pytest.mark.parametrize("T,E,k,d", [(7, 5, 2, 8)])
def test_dense_router_backward_reduces_to_the_sparse_one(T, E, k, d):
    rng = np.random.default_rng(4)
    z = rng.standard_normal((T, E)).astype(np.float32)
    idx, gates = route.topk_gates(z, k)
    P = route.permutation(idx, E)
    dl = route.route_backward(rng.standard_normal((T, k)).astype(np.float32), gates, idx, E)
    x = rng.integers(0x3F00, 0x4000, (T, d)).astype(np.uint16)
    w = rng.integers(0x3F00, 0x4000, (E, d)).astype(np.uint16)
    dxp = rng.standard_normal((T * k, d)).astype(np.float32)
    assert np.allclose(router.weight_grad_dense(x, dl)[0], router.weight_grad(x, dl, idx), rtol=1e-13)
    from oracle import formats as fmt
    dense, _ = router.unpermute_sum_dense(dxp, P["inv_perm"], T, k, dl, w)
    sparse = fmt.bf16_to_f32(router.unpermute_sum_router(dxp, P["inv_perm"], T, k, dl, idx, w)).astype(np.float64)
    assert np.allclose(sparse, dense, rtol=2.0 ** -7, atol=1e-5)


def test_rows_that_are_not_finite():
    """A NaN or +infinity makes its row NaN whatever else is in it; -infinities are zeros, also where there is nothing else."""
    inf, nan = np.inf, np.nan
    z = np.float32([[nan, nan, nan], [-inf, nan, -inf], [0, 1, nan], [0, inf, -inf], [-inf] * 3, [-inf, 0, 0]])
    with np.errstate(invalid="ignore"):
        r = balance.balance_loss(z, np.zeros((6, 1), int), seg_off=range(7))
        g = balance.balance_grad(np.ones(6), z, r["counts"], r["tokens"], 1, seg_off=range(7))
    assert np.isnan(r["probs"][:4]).all() and np.isnan(r["loss"][:4]).all() and np.isnan(g[:4]).all()
    assert r["probs"][4:].tolist() == [[0, 0, 0], [0, 0.5, 0.5]] and r["loss"][4:].tolist() == [0, 0] and not g[4:].any()
