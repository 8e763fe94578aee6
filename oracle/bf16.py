"""The expert layer in BF16, in float64 (test infrastructure).

The pages keep some activations in BF16 and measure their 4-bit rates against
BF16 (lhc.media page, paragraph on the precisions that remain; fourweekmba.com
page, the hardware table); they do not describe an unquantised expert layer.
The readings taken are the usual forms: experts act(x W^T + b), or gated
act(x W_g^T + b_g) (x W_u^T + b_u); SiLU, or GELU by its tanh form; inverted
dropout with the random words of the stochastic rounding.

Operands are float64 arrays holding bf16 values.  Each product also returns
the sum of its terms' magnitudes, which the tolerances of the tests scale with.
"""
import numpy as np

from . import srhash

NONE, SILU, GELU = 0, 1, 2
_C = 2.0 * np.sqrt(2.0 / np.pi)


def _sigmoid(p):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-p))


def act(kind, x):
    """act(x) and act'(x)."""
    x = np.asarray(x, dtype=np.float64)
    if kind == NONE:
        return x.copy(), np.ones_like(x)
    p, dp = (x, 1.0) if kind == SILU else (_C * (x + 0.044715 * x ** 3), _C * (1.0 + 0.134145 * x * x))
    t = _sigmoid(p)
    s = t * _sigmoid(-p)
    with np.errstate(invalid="ignore"):
        return np.where(np.isneginf(x), -0.0, x * t), np.where(s == 0.0, t, t + x * s * dp)


def rows(x, row_map=None, div=1):
    """The gathered operand."""
    return x if row_map is None else x[np.asarray(row_map, dtype=np.int64) // div]


def groups(off):
    off = np.asarray(off, dtype=np.int64)
    return [(e, int(a), int(b)) for e, (a, b) in enumerate(zip(off[:-1], off[1:])) if b > a]


def product(a, w, off, transpose):
    """z[r] = a[r] . w[e]^T (transpose) or a[r] . w[e], and sum |a| |w|; NaN in rows of no expert."""
    n = w.shape[1] if transpose else w.shape[2]
    z, m = np.full((a.shape[0], n), np.nan), np.full((a.shape[0], n), np.nan)
    for e, r0, r1 in groups(off):
        b = w[e].T if transpose else w[e]
        z[r0:r1] = a[r0:r1] @ b
        m[r0:r1] = np.abs(a[r0:r1]) @ np.abs(b)
    return z, m


def per_row(v, off, M):
    """Expert values v [E, n] spread over the rows (0 in rows of no expert)."""
    out = np.zeros((M,) + v.shape[1:])
    for e, r0, r1 in groups(off):
        out[r0:r1] = v[e]
    return out


def wgrad(dy, a, off):
    """dw [E, N, K] and the magnitudes' sums."""
    E = len(off) - 1
    dw, m = np.zeros((E, dy.shape[1], a.shape[1])), np.zeros((E, dy.shape[1], a.shape[1]))
    for e, r0, r1 in groups(off):
        dw[e] = dy[r0:r1].T @ a[r0:r1]
        m[e] = np.abs(dy[r0:r1]).T @ np.abs(a[r0:r1])
    return dw, m


def keep_mask(T, d, p, seed, stream_id):
    """(kept [T, d] bool, the factor of a kept value)."""
    q = int(np.rint((1.0 - p) * 65536.0))
    r = srhash.random16(seed, stream_id, np.arange(T * d, dtype=np.uint64))
    return (r < q).reshape(T, d), 65536.0 / q if q else 0.0


def combine_dropout(yp, gates, inv_perm, p, seed, stream_id, residual=None):
    T, k = gates.shape
    acc = (gates[:, :, None] * yp[np.asarray(inv_perm).reshape(T, k)]).sum(axis=1)
    keep, f = keep_mask(T, yp.shape[1], p, seed, stream_id)
    y = np.where(keep, acc * f, 0.0)
    return y if residual is None else y + residual


def layer(x, w_up, w_down, logits_perm, k, act_kind, b_up=None, b_down=None):
    """Routed experts on given routing (dict off, perm, inv_perm, gates): Yp and the intermediates."""
    r = logits_perm
    a = rows(x, r["perm"], k)
    gated = w_up.ndim == 4
    E, F = w_up.shape[0], w_up.shape[-2]
    z, _ = product(a, w_up.reshape(E, -1, w_up.shape[-1]), r["off"], True)
    if b_up is not None:
        z = z + per_row(b_up.reshape(E, -1), r["off"], len(a))
    h = act(act_kind, z[:, :F])[0] * z[:, F:] if gated else act(act_kind, z)[0]
    yp, _ = product(h, w_down, r["off"], True)
    if b_down is not None:
        yp = yp + per_row(b_down, r["off"], len(a))
    return dict(z=z, h=h, yp=yp)
