"""Operands and error bounds of the BF16 expert products' tests."""
import numpy as np
import torch

from oracle import bf16 as ob

U = 2.0 ** -24
L_ACT = 1.13          # the largest slope of SiLU (1.10) and GELU (1.129)


def bf(x):
    """float64 array of the bf16 values of x, and the CPU tensor."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t


def offsets(m_list, lead=0):
    return np.concatenate([[0], np.cumsum(m_list)]).astype(np.int64) + lead


def z_err(K, mag):
    """Exact products; a float32 accumulation of K terms rounds at most K times, each by at most one
    unit (2**-23, a cut as well as a rounding) of a partial sum that is at most the terms' magnitude."""
    return K * 2.0 ** -23 * mag


def act_parts(kind, x):
    """act, act', and the bounds of their evaluation's error in float32.

    t = sigmoid(p) has a relative error of (|p| + 8) 2**-23: the exponent's argument is rounded (|p|
    2**-24, and p itself for GELU by as much again), exp2, the sum and the reciprocal cost a unit each.
    act = x t adds a rounding.  act' = t + x s p', s = t (1 - t): where t > 1/2 the difference 1 - t
    has an absolute error of a unit of 1 (and s is taken as 0 below half of one), times |x p'|, which
    is at most 20 (SiLU: 1 - t vanishes beyond x = 18) or 4 * 4 (GELU); elsewhere s is as exact as t."""
    f, d = ob.act(kind, x)
    if kind == ob.NONE:
        return f, d, np.zeros_like(f), np.zeros_like(d)
    x = np.asarray(x, dtype=np.float64)
    p, dp = (x, np.ones_like(x)) if kind == ob.SILU else (ob._C * (x + 0.044715 * x ** 3), ob._C * (1 + 0.134145 * x * x))
    t = ob._sigmoid(p)
    s = t * ob._sigmoid(-p)
    rel = (2 * np.abs(p) + 8) * 2.0 ** -23
    tiny = 2.0 ** -118                       # where 1 + exp2 overflows: |x| 2**-126 and less
    ef = np.abs(f) * rel + tiny
    ed = t * rel + np.abs(x * s * dp) * 2 * rel + np.where(t > 0.5, np.minimum(np.abs(x * dp), 20.0) * 2.0 ** -22, 0.0) + tiny
    return f, d, ef, ed


def check(got, exact, err, bf16, what=""):
    """|got - exact| <= err and half a unit of the output's type at |exact| + err, NaN where exact is."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == exact.shape, (what, got.shape, exact.shape)
    a = np.maximum(np.abs(exact) + err, 2.0 ** -126)
    lim = err * (1 + 2.0 ** -20) + 0.5 * np.exp2(np.floor(np.log2(a)) - (7 if bf16 else 23))
    bad = ~(np.abs(got - exact) <= lim)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off; first at {np.argwhere(bad)[0]}: {got[bad][0]} for {exact[bad][0]}, bound {lim[bad][0]}"


class Case:
    """Random operands of experts with m_list rows: gathered or not."""

    def __init__(self, m_list, n, k, seed, mapped=False, div=2, lead=0, tail=0, dup=False):
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.off = offsets(m_list, lead)
        self.M = int(self.off[-1]) + tail
        self.E, self.n, self.k = len(m_list), n, k
        self.div = div if mapped else 1
        self.map = None
        rows = self.M
        if mapped:
            rows = (self.M + div - 1) // div + 1
            self.map = (rng.integers(0, rows * div, self.M) if dup else rng.permutation(rows * div)[:self.M]).astype(np.int32)
        self.rows = rows
        self.live = np.zeros(self.M, bool)
        self.live[self.off[0]:self.off[-1]] = True

    def bf(self, *shape, std=1.0):
        v, t = bf(self.rng.standard_normal(shape) * std)
        return v, t.cuda()

    def f32(self, *shape, std=1.0):
        a = (self.rng.standard_normal(shape) * std).astype(np.float32)
        return a.astype(np.float64), torch.from_numpy(a).cuda()

    def gpu_off(self):
        return torch.from_numpy(self.off.astype(np.int32)).cuda()

    def gpu_map(self):
        return None if self.map is None else torch.from_numpy(self.map).cuda()

    def gather(self, x):
        return ob.rows(x, self.map, self.div)

    def scale_of(self, s):
        """A row scale's values by row of the product (ones without)."""
        if s is None:
            return np.ones((self.M, 1))
        return (s if self.map is None else s[self.map])[:, None]
