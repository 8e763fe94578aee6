"""Edges of the balance loss, the dense router backward, MXFP4 quantisation and
its transposed requantisation: logits and gradients that are not finite or tiny,
launch sizes, a dispatch to no rows, padded offsets outside the outputs."""
import ctypes

import numpy as np
import pytest
import torch

from gpu_helpers import bf16_from_bits, cuda_f32, cuda_i32, to_np
from oracle import balance as ob
from oracle import formats as fmt

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import precision_moe_numerics_quant_amd as m4

U = 2.0 ** -24


# -------------------------------------------------------------- balance loss

@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E", [1, 2, 8, 9, 64, 130, 384, 1024])
def test_balance_rows_that_are_not_finite(E, bias):
    """A row with a NaN or +infinity anywhere, whatever else it holds, has NaN probabilities, loss and gradient; a row
    of -infinities has zeros; every other row is as ever.  One segment per row, then one for all."""
    rng = np.random.default_rng(E)
    T, k, inf, nan = 14, 1, np.inf, np.nan
    z = rng.standard_normal((T, E)).astype(np.float32)
    b = rng.standard_normal(E).astype(np.float32) if bias else None
    z[1] = nan
    z[2], z[2, E // 2] = -inf, nan
    z[3, E - 1] = nan
    z[4, 0] = inf
    z[5], z[5, E - 1] = -inf, inf
    z[6] = inf
    z[7] = -inf
    z[8, :E - 1] = -inf                         # one finite value (E = 1: an ordinary row)
    z[9], z[9, 0] = inf, -inf
    z[10, 0], z[10, E - 1] = -inf, nan
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    for seg in (np.arange(T + 1), [0, T]):
        kw = dict(bias=None if b is None else cuda_f32(b), seg_off=cuda_i32(seg))
        r = m4.moe_balance_loss(cuda_f32(z), cuda_i32(idx), **kw)
        with np.errstate(invalid="ignore"):
            o = ob.balance_loss(z, idx, b, None, seg)
            dl = rng.standard_normal(len(seg) - 1).astype(np.float32)
            g = ob.balance_grad(dl, z, o["counts"], o["tokens"], k, b, None, seg)
        assert np.array_equal(to_np(r["counts"]), o["counts"]) and np.array_equal(to_np(r["tokens"]), o["tokens"])
        got = to_np(m4.moe_balance_loss_backward(cuda_f32(dl), cuda_f32(z), r["counts"], r["tokens"], k, **kw))
        # the argument of the exponential rounds twice at its magnitude (below 16 here), the exponential by two units,
        # the sum of E terms E / 64 + 6 times, a reciprocal and a product; then 14 terms and E products of the loss
        tol = (2 * 16 + E / 64 + 6 + 8 + 16 + E + 6) * U
        for name in ("probs", "loss"):
            a, w = to_np(r[name]).astype(np.float64), o[name]
            assert np.array_equal(np.isnan(a), np.isnan(w)), name
            ok = ~np.isnan(w)
            assert (np.abs(a - w)[ok] <= tol * np.abs(w)[ok]).all(), name
        assert np.array_equal(np.isnan(got), np.isnan(g))
        # two terms of at most dloss E / (k n^2) max(c) each with p's error
        lim = 4 * tol * np.abs(dl).max() * E * max(1, o["counts"].max())
        assert (np.abs(got - g)[~np.isnan(g)] <= lim).all()


def test_balance_gradient_of_more_tokens_than_one_grid_row():
    """2**26 + 5 tokens: more than 2**32 threads of one wave per token.  Rows repeat a pattern of 1024, whose results
    are checked in float64; equal rows have equal bits wherever they are."""
    P, T, E, k = 1024, (1 << 26) + 5, 2, 1
    rng = np.random.default_rng(26)
    zp = rng.standard_normal((P, E)).astype(np.float32)
    ip = (zp[:, 1] > zp[:, 0]).astype(np.int32)[:, None]
    rep = lambda a: torch.cat([a.repeat(T // P, 1), a[:T % P]])
    z, idx = rep(cuda_f32(zp)), rep(cuda_i32(ip))
    r = m4.moe_balance_loss(z, idx)
    p = ob.softmax(zp)
    full, rest = T // P, T % P
    count = np.bincount(ip[:, 0], minlength=E) * full + np.bincount(ip[:rest, 0], minlength=E)
    mean = (p.sum(0) * full + p[:rest].sum(0)) / T
    assert np.array_equal(to_np(r["counts"])[0], count) and int(r["tokens"][0]) == T
    # sums of positive terms: 4 tokens in turn per wave, 16 waves, 2**20 chunks in 32 shares, the shares; each softmax
    # is good to 32 units here
    tol = (4 + 16 + (1 << 15) + 1 + 32 + 32 + 8) * U
    assert (np.abs(to_np(r["probs"])[0] - mean) <= tol * mean).all()
    loss = E / (k * T) * (count * mean).sum()
    assert abs(float(r["loss"][0]) - loss) <= (tol + 8 * U) * loss
    dl = torch.full((1,), 1e6, device="cuda")
    g = m4.moe_balance_loss_backward(dl, z, r["counts"], r["tokens"], k)
    c = count.astype(np.float64)
    want = 1e6 * E / (k * float(T) ** 2) * p * (c[None, :] - (p @ c)[:, None])
    dev = np.abs(c - c.mean()).max()
    lim = 1e6 * E / (k * float(T) ** 2) * p * 2 * dev * (3 * 32 + 16) * U
    # (the counts' difference from their mean: an exact integer less a rounded k n / E, half a unit of 2**25)
    lim = lim + 1e6 * E / (k * float(T) ** 2) * p * 4
    assert (np.abs(to_np(g[:P]) - want) <= lim).all()
    assert torch.equal(g[:full * P].view(full, P, E), g[:P].expand(full, P, E)) and torch.equal(g[full * P:], g[:rest])


# -------------------------------------------------------------- dense router

def test_dense_router_infinite_gradients():
    """An infinite dlogits value gives infinite results of the products' signs, two of opposite signs a NaN; a NaN of
    any payload gives NaN."""
    T, E, d, k = 130, 40, 64, 2
    rng = np.random.default_rng(3)
    dz = rng.standard_normal((T, E)).astype(np.float32)
    dz[3, 5], dz[129, 39] = np.inf, -np.inf
    dz[64, 7], dz[64, 8] = np.inf, -np.inf
    dz.view(np.uint32)[70, 20], dz.view(np.uint32)[71, 21] = 0x7F800001, 0xFFFFFFFF
    sign = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    w = fmt.f64_to_bf16((1 + rng.random((E, d))) * sign)
    x = fmt.f64_to_bf16((1 + rng.random((T, d))) * sign)
    dx = m4.moe_unpermute_sum_router_dense(cuda_f32(np.ones((T * k, d), np.float32)), cuda_i32(rng.permutation(T * k).astype(np.int32)),
                                           T, k, cuda_f32(dz), bf16_from_bits(w)).float().cpu().numpy()
    assert np.array_equal(dx[3], np.inf * sign) and np.array_equal(dx[129], -np.inf * sign)
    assert np.isnan(dx[[64, 70, 71]]).all()
    assert np.isfinite(dx[~np.isin(np.arange(T), [3, 64, 70, 71, 129])]).all()
    dw = to_np(m4.moe_router_wgrad_dense(bf16_from_bits(x), cuda_f32(dz)))
    for e, s in ((5, 1), (7, 1), (8, -1), (39, -1)):
        assert np.array_equal(dw[e], s * np.inf * sign), e
    assert np.isnan(dw[[20, 21]]).all()
    assert np.isfinite(dw[~np.isin(np.arange(E), [5, 7, 8, 20, 21, 39])]).all()


def test_dense_router_split_of_small_gradients():
    """One-hot x: dW is dz itself, exactly from 2**-110 on (the lowest significand bit is then bf16's smallest
    subnormal, 2**-133); below, short of it by less than 2**-133."""
    rng = np.random.default_rng(8)
    eye = bf16_from_bits(fmt.f64_to_bf16(np.eye(64)))
    m = rng.integers(1 << 23, 1 << 24, (64, 64)).astype(np.float64) * np.where(rng.random((64, 64)) < 0.5, -1, 1)
    dz = (m * np.exp2(rng.integers(-133, -110, (64, 64)))).astype(np.float32)
    assert np.array_equal(to_np(m4.moe_router_wgrad_dense(eye, cuda_f32(dz))), dz.T)
    dz = (m * np.exp2(rng.integers(-149, -133, (64, 64)))).astype(np.float32)
    got = to_np(m4.moe_router_wgrad_dense(eye, cuda_f32(dz))).astype(np.float64)
    assert (np.abs(got - dz.T.astype(np.float64)) < 2.0 ** -133).all()


# --------------------------------------------------------------------- MXFP4

def test_quant_dispatch_without_output_rows_reports():
    """No output rows at all: every entry is outside and reported."""
    x = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    out = (torch.empty((0, 32), dtype=torch.uint8, device="cuda"), torch.empty((0, 2), dtype=torch.uint8, device="cuda"))
    m4.mxfp4_quant(x, out_map=cuda_i32([0, 1, 2]), out=out)
    with pytest.raises(m4.Moe4DeviceError, match="clamped"):
        m4.moe4_debug_check()
    m4.mxfp4_quant(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), out_map=cuda_i32([]), out=out)
    m4.moe4_debug_check()


@pytest.mark.parametrize("offp", [[0, 1 << 20, 64], [-64, 32, 64], [0, 96, 64], [0, 5, 64], [0, 32, 96], [0, 32, -32]])
def test_requant_padded_offsets_outside(offp):
    """Padded offsets that are not ascending multiples of 32 up to max_padded_rows: reported, and nothing written around
    the outputs (offsets that end below zero leave no blocks at all)."""
    C, mpr, guard = 544, 64, 1 << 16
    q, s = torch.zeros((40, C // 2), dtype=torch.uint8, device="cuda"), torch.full((40, C // 32), 127, dtype=torch.uint8, device="cuda")
    oc, os_ = (torch.full((2 * guard + n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (C * mpr, C * mpr // 32))
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    off, op = cuda_i32([0, 20, 40]), cuda_i32(offp)
    rc = m4.lib().mxfp8_requant_mx4_sr_T(ptr(q), ptr(s), 40, C, ptr(off), ptr(op), 2, mpr, 1, 2, 0, ptr(oc[guard:]), ptr(os_[guard:]),
                                         ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    if offp[-1] > 0:
        with pytest.raises(m4.Moe4DeviceError, match="offset"):
            m4.moe4_debug_check()
    for t in (oc, os_):
        assert (t[:guard] == 0x5A).all() and (t[-guard:] == 0x5A).all()
