"""The router's balance loss and its gradient in float64 (test infrastructure).

The pages route each token to 8 of 384 experts (fourweekmba.com page,
"Update") and do not say how the load is kept even.  The reading taken: the
usual auxiliary loss, per segment s of tokens with n_s unmasked tokens,
  counts[s, e] = assignments to e, probs[s, e] = mean of softmax(z[t])[e],
  loss[s] = E / (k n_s) sum_e counts[s, e] probs[s, e],
z = logits + bias (added in float32, as the routing does); the counts are
constants of the gradient.
"""
import numpy as np


def softmax(z):
    z = np.asarray(z, dtype=np.float64)
    m = z.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.exp(z - m)
    p[np.isneginf(m[:, 0])] = 0.0                    # a row of -infinities
    s = p.sum(axis=1, keepdims=True)
    return np.divide(p, s, out=np.zeros_like(p), where=s != 0)


def _z(logits, bias):
    z = np.asarray(logits, dtype=np.float32)
    return z if bias is None else (z + np.asarray(bias, dtype=np.float32)).astype(np.float32)


def _segments(T, seg_off):
    off = [0, T] if seg_off is None else [int(v) for v in seg_off]
    return list(zip(off[:-1], off[1:]))


def _live(T, mask):
    return np.ones(T, dtype=bool) if mask is None else np.asarray(mask).astype(bool)


def balance_loss(logits, idx, bias=None, mask=None, seg_off=None):
    """dict(loss [S], counts [S, E], tokens [S], probs [S, E])."""
    T, E = np.asarray(logits).shape
    idx = np.asarray(idx, dtype=np.int64)
    k = idx.shape[1]
    live = _live(T, mask)
    z = _z(logits, bias)
    loss, counts, tokens, probs = [], [], [], []
    for a, b in _segments(T, seg_off):
        on = np.flatnonzero(live[a:b]) + a
        n = len(on)
        c = np.bincount(idx[on].reshape(-1), minlength=E)
        m = softmax(z[on]).sum(axis=0) / n if n else np.zeros(E)
        loss.append(E / (k * n) * float((c * m).sum()) if n else 0.0)
        counts.append(c)
        tokens.append(n)
        probs.append(m)
    return dict(loss=np.array(loss), counts=np.array(counts), tokens=np.array(tokens), probs=np.array(probs))


def balance_grad(dloss, logits, counts, tokens, k, bias=None, mask=None, seg_off=None):
    """d(sum_s dloss[s] loss[s]) / dlogits [T, E] (zeros for masked tokens and tokens outside the segments)."""
    T, E = np.asarray(logits).shape
    live = _live(T, mask)
    z = _z(logits, bias)
    g = np.zeros((T, E))
    for s, (a, b) in enumerate(_segments(T, seg_off)):
        on = np.flatnonzero(live[a:b]) + a
        n = int(tokens[s])
        if not len(on) or not n:
            continue
        p = softmax(z[on])
        c = np.asarray(counts[s], dtype=np.float64)
        g[on] = float(dloss[s]) * E / (k * n * n) * p * (c[None, :] - (p @ c)[:, None])
    return g
