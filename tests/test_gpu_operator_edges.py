"""Edges of the balance loss, the dense router backward, MXFP4 quantisation,
its transposed requantisation and the grouped MXFP4 product: logits and
gradients that are not finite, launch sizes, long contractions through the
product's rings, stores next to other rows, scale bytes at the requantisation's
borders, offsets past 32 bits."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from gpu_helpers import assert_bytes_equal, bf16_from_bits, cuda_f32, cuda_i32, cuda_u8, to_np
from oracle import balance as ob
from oracle import formats as fmt
from oracle import gemm as og
from oracle import mxfp4
from oracle import mxfp8 as mx
from oracle import router
from oracle import silu as osilu
from oracle import srhash

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import precision_moe_numerics_quant_amd as m4
    from precision_moe_numerics_quant_amd import layer

U = 2.0 ** -24
LAYOUTS = {0: mx.SF_ROWS, 1: mx.SF_BLOCKS}


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


def test_dense_router_many_slots_of_a_large_batch():
    """64-row tiles with more slots than are in flight at a time, E and d inside a tile."""
    T, E, k, d = 4100, 33, 12, 1028
    rng = np.random.default_rng(12)
    inv = rng.permutation(T * k).astype(np.int32)
    dxp = (1e-2 * rng.standard_normal((T * k, d))).astype(np.float32)
    dz = rng.standard_normal((T, E)).astype(np.float32)
    wb = fmt.f64_to_bf16(0.05 * rng.standard_normal((E, d)))
    dx = m4.moe_unpermute_sum_router_dense(cuda_f32(dxp), cuda_i32(inv), T, k, cuda_f32(dz), bf16_from_bits(wb))
    exact, mag = router.unpermute_sum_dense(dxp, inv, T, k, dz, wb)
    # exact products; k + 3 E additions of float32, cut or rounded, then half a bf16 unit
    slack = (k + 3 * E + 2) * 2 * U * mag
    lim = slack + 2.0 ** -8 * np.exp2(np.floor(np.log2(np.abs(exact) + slack + 1e-300)))
    assert (np.abs(dx.float().cpu().numpy() - exact) <= lim).all()


@pytest.mark.parametrize("variant", ["nvfp4", "mxfp8", "mxfp4"])
def test_layer_balance_without_the_router(variant):
    """Each variant of the layer on given logits: dlogits gains the balance gradient and nothing else changes."""
    inp, c = synth.config_inputs(1, device="cpu"), synth.CONFIGS[1]
    T, E, k = c["T"], c["E"], c["k"]
    x, wu, wd, lg, dy = (inp[n].cuda() for n in ("x", "w_up", "w_down", "logits", "dy"))
    f, b = dict(nvfp4=(layer.forward, layer.backward), mxfp8=(layer.forward_mx, layer.backward_mx),
                mxfp4=(layer.forward_mx4, layer.backward_mx4))[variant]
    bias = torch.linspace(-0.2, 0.2, E, device="cuda")
    plain = f(x, wu, wd, lg, k, bias=bias)
    fw = f(x, wu, wd, lg, k, bias=bias, balance=True)
    assert torch.equal(plain["y"], fw["y"])
    o = ob.balance_loss(inp["logits"].numpy(), to_np(fw["route"]["idx"]), to_np(bias))
    assert np.array_equal(to_np(fw["balance"]["counts"]), o["counts"])
    coef = torch.full((1,), 0.5, device="cuda")
    ref, got = b(plain, dy), b(fw, dy, dbalance=coef)
    for n in ("dx", "dW_up", "dW_down", "dg"):
        assert torch.equal(ref[n], got[n]), n
    g = ob.balance_grad([0.5], inp["logits"].numpy(), o["counts"], o["tokens"], k, to_np(bias))
    p, cc = ob.softmax(inp["logits"].numpy() + to_np(bias)), np.abs(o["counts"][0] - k * T / E)
    span = 2 * (np.abs(inp["logits"].numpy()).max() + 0.2)
    # the softmax (its argument's two roundings, E terms, a handful more) in both terms of f p (c - sum p c), then the sum
    eps = (2 * span + E / 64 + 14) * U
    lim = 0.5 * E / (k * T ** 2) * p * (cc + (p @ cc)[:, None]) * (3 * eps + 16 * U)
    r = to_np(ref["dlogits"]).astype(np.float64)
    assert (np.abs(to_np(got["dlogits"]) - (r + g)) <= lim + 2 * U * (np.abs(r) + np.abs(g))).all() and np.abs(g).max() > 0


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


@pytest.mark.parametrize("copies", [1, 11])
@pytest.mark.parametrize("silu", [False, True])
def test_quant_dispatch_of_many_copies_and_silu(copies, silu):
    """A map with more copies than are looked up at a time, and the map together with SiLU."""
    R, C = 70, 544
    rng = np.random.default_rng(copies)
    x = fmt.f64_to_bf16(3 * rng.standard_normal((R, C)))
    to = rng.permutation(R * copies).astype(np.int32)
    got = m4.mxfp4_quant(bf16_from_bits(x), m4.PRE_SILU if silu else m4.PRE_NONE, cuda_i32(to), copies)
    q, s = mxfp4.quantize(osilu.silu_f32(x) if silu else fmt.bf16_to_f32(x))
    inv = np.argsort(to) // copies
    assert_bytes_equal(to_np(got[0]), q[inv], "codes")
    assert_bytes_equal(to_np(got[1]), s[inv], "scales")


def test_empty_batch():
    """No rows: an empty dispatch, and the MXFP4 forward with its balance loss."""
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    for silu in (m4.PRE_NONE, m4.PRE_SILU):
        codes, sf = m4.mxfp4_quant(x, silu, out_map=cuda_i32([]), copies=8)
        assert codes.shape == (0, 32) and sf.shape == (0, 2)
    inp, c = synth.config_inputs(1, device="cpu"), synth.CONFIGS[1]
    fw = layer.forward_mx4(inp["x"][:0].cuda(), inp["w_up"].cuda(), inp["w_down"].cuda(), inp["logits"][:0].cuda(), c["k"], balance=True)
    assert fw["y"].shape == (0, c["d"]) and not fw["balance"]["loss"].any() and not fw["balance"]["tokens"].any()
    m4.moe4_debug_check()


def _requant_check(q, s, off, lay, what):
    offp = mx.padded_offsets(off)
    got = m4.mxfp8_requant_mx4_sr_T(cuda_u8(q), cuda_u8(s), cuda_i32(off), cuda_i32(offp), 7, 33, int(offp[-1]), lay)
    want = mxfp4.requant_sr_t(q, s, off, 7, 33, LAYOUTS[lay])
    assert_bytes_equal(to_np(got[1]), want[1], what + " scales")
    assert_bytes_equal(to_np(got[0]), want[0], what + " codes")


BORDERS = ["all 20", "all 251", "20 and 251", "20 .. 251", "19 among 127", "252 among 127", "254 among 20", "zero rows", "zero blocks"]


@pytest.mark.parametrize("lay", [0, 1])
@pytest.mark.parametrize("what", BORDERS)
def test_requant_scales_at_the_borders(what, lay):
    """Bytes at the ends of [20, 251], blocks that mix both ends (v / scale down to 2**-233), single rows just outside,
    and rows and blocks of zeros (scale byte 0) among ordinary ones; more than 512 columns, a partial last block."""
    rng = np.random.default_rng(BORDERS.index(what))
    off = np.array([0, 70, 70, 103, 167])
    R, C = 167, 1056
    q = rng.integers(0, 256, (R, C // 2), dtype=np.uint8)
    s = np.full((R, C // 32), 127, np.uint8)
    if what == "all 20":
        s[:] = 20
    elif what == "all 251":
        s[:] = 251
    elif what == "20 and 251":
        s[0::2], s[1::2] = 20, 251
    elif what == "20 .. 251":
        s = rng.integers(20, 252, (R, C // 32), dtype=np.uint8)
    elif what == "19 among 127":
        s[[3, 90]] = 19
    elif what == "252 among 127":
        s[[3, 90]] = 252
    elif what == "254 among 20":
        s[:] = 20
        s[[3, 90]] = 254
    elif what == "zero rows":
        q[::10], s[::10] = 0, 0
    else:
        q[5, 32:48], s[5, 2] = 0x88, 0             # one block of negative zeros
        q[120, :16], s[120, 0] = 0, 0
    _requant_check(q, s, off, lay, what)


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


# ------------------------------------------------------------------- product

def _ints(M, off, E, N, K, seed):
    """Random codes under scales 2**-1 .. 2**1: products are multiples of 2**-4 below 144, so every partial sum of up to
    7281 of them is exact in float32, in any order."""
    assert K <= 7281
    rng = np.random.default_rng(seed)
    a, b = rng.integers(0, 256, (M, K // 2), dtype=np.uint8), rng.integers(0, 256, (E * N, K // 2), dtype=np.uint8)
    sa, sb = rng.integers(126, 129, (M, K // 32), dtype=np.uint8), rng.integers(126, 129, (E * N, K // 32), dtype=np.uint8)
    want = og.grouped_nt(mxfp4.dequant(a, sa), mxfp4.dequant(b, sb).reshape(E, N, K), off)
    return (a, sa), (b, sb), want


def _product(qa, qb, off, E, N, K, dt):
    return m4.moe_grouped_gemm_mx4(cuda_u8(qa[0]), cuda_u8(qa[1]), cuda_u8(qb[0]).view(E, N, K // 2),
                                   cuda_u8(qb[1]).view(E, N, K // 32), cuda_i32(off), dt)


def _check_exact(c, want):
    if c.dtype == torch.bfloat16:
        assert_bytes_equal(to_np(c), fmt.f64_to_bf16(want), "bf16")
    else:
        assert np.array_equal(to_np(c).astype(np.float64), want)


MANY = [0, 137, 1, 400, 0, 290, 128, 31, 256, 3] * 4
LONG = [([700, 1500, 3], 384, 2048), ([700, 1500, 3], 160, 2080), ([700, 1500, 3], 1024, 2048), ([130, 0, 700], 544, 4096),
        (MANY, 2560, 1024), (MANY, 1280, 1056), ([3 * m for m in MANY], 384, 1024), ([2100, 700, 1, 0, 900], 32, 1504)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M_list,N,K", LONG)
def test_gemm_long_contractions_and_many_tiles(M_list, N, K, dt):
    """Every stage and scale buffer of the tiled kernels refilled (four slabs of 256 and more per tile), up to three
    tiles per workgroup, tiles that end after one row next to full ones: exact, and the same bits from a second call."""
    E = len(M_list)
    off = np.concatenate([[0], np.cumsum(M_list)])
    qa, qb, want = _ints(int(off[-1]), off, E, N, K, N + K)
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    c = _product(qa, qb, off, E, N, K, t)
    _check_exact(c, want)
    assert torch.equal(c, _product(qa, qb, off, E, N, K, t))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M_list,N,K", [([40, 0, 23], 96, 160), ([300, 0, 131, 1, 257], 160, 544), ([300, 0, 131, 1, 257], 384, 1024),
                                        ([300, 0, 131, 1, 257], 544, 1024), (MANY, 2592, 512)])
def test_gemm_writes_its_rows_only(M_list, N, K, dt):
    """The few-rows kernel and the tiled ones (128 columns without and with pairs of scales, 256 columns): expert_off[0]
    above zero, rows behind the last expert, C in the middle of a larger buffer; nothing but the experts' rows changes.
    The other rows of A are NaN throughout."""
    E, lead, tail, guard = len(M_list), 5, 9, 4096
    off = lead + np.concatenate([[0], np.cumsum(M_list)])
    M = int(off[-1]) + tail
    qa, qb, want = _ints(M, off, E, N, K, N + K)
    for s in qa:
        s[:lead] = 0xFF
        s[off[-1]:] = 0xFF
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    dev = [cuda_u8(v) for v in (*qa, *qb)] + [cuda_i32(off)]
    bufs = []
    for _ in range(2):
        buf = torch.full((guard + M * N + guard,), 7.0, dtype=t, device="cuda")
        rc = m4.lib().moe_grouped_gemm_mx4(*(ctypes.c_void_p(v.data_ptr()) for v in dev), E, M, N, K,
                                           ctypes.c_void_p(buf[guard:].data_ptr()), m4.BF16 if dt == "bf16" else m4.F32,
                                           ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert rc == 0
        bufs.append(buf)
    assert torch.equal(bufs[0], bufs[1])
    c = bufs[0][guard:guard + M * N].view(M, N)
    assert (bufs[0][:guard] == 7).all() and (bufs[0][guard + M * N:] == 7).all()
    assert (c[:lead] == 7).all() and (c[off[-1]:] == 7).all()
    _check_exact(c[lead:off[-1]], want[lead:off[-1]])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gemm_training_shape_sampled(dt):
    """131072 skewed rows of 384 experts, N = 1536, K = 4096, operands whose sums are exact: whole rows at the starts
    and ends of experts and between."""
    E, M, N, K = 384, 131072, 1536, 4096
    g = torch.Generator(device="cuda").manual_seed(5)
    a, b = (torch.randint(0, 256, (n, K // 2), dtype=torch.uint8, device="cuda", generator=g) for n in (M, E * N))
    sa, sb = (torch.randint(126, 129, (n, K // 32), dtype=torch.uint8, device="cuda", generator=g) for n in (M, E * N))
    share = 1.0 / np.arange(1, E + 1) ** 1.1
    sizes = np.floor(M * share / share.sum()).astype(int)
    sizes[300:] = 0
    sizes[0] += M - sizes.sum()
    off = np.concatenate([[0], np.cumsum(np.random.default_rng(1).permutation(sizes))])
    c = m4.moe_grouped_gemm_mx4(a, sa, b.view(E, N, -1), sb.view(E, N, -1), cuda_i32(off), torch.bfloat16 if dt == "bf16" else torch.float32)
    rows = np.unique(np.concatenate([np.linspace(0, M - 1, 12).astype(int), off[50:56], off[50:56] - 1]))
    for i in rows[(rows >= 0) & (rows < M)]:
        e = int(np.searchsorted(off, i, side="right") - 1)
        A = mxfp4.dequant(to_np(a[i:i + 1]), to_np(sa[i:i + 1]))
        B = mxfp4.dequant(to_np(b[e * N:(e + 1) * N]), to_np(sb[e * N:(e + 1) * N]))
        _check_exact(c[i:i + 1], A @ B.T)


FEW = [0] * 91 + [1, 2, 0, 3, 1] + [0] * 200 + [2, 1] + [0] * 86           # 10 rows among 384 experts
ONE_LONG = [i % 3 for i in range(90)] + [0, 150, 17]                         # one expert of three blocks of 64 rows


@pytest.mark.parametrize("M_list,N,K", [(FEW, 96, k) for k in (512, 1536, 2048, 2560, 4096, 5120, 7168)] +
                         [(FEW, 64, k) for k in (544, 1056, 2080, 4128, 5152)] +
                         [(ONE_LONG, 96, 1536), (ONE_LONG, 32, 160), (ONE_LONG, 64, 7168), (ONE_LONG, 32, 5152)])
def test_gemm_few_rows_of_many_experts(M_list, N, K):
    """The few-rows kernel with more experts than lanes, at every number of K steps that a wave holds and past it
    (K > 4096: weights read again for every 16 rows), K with and without whole steps."""
    E = len(M_list)
    off = np.concatenate([[0], np.cumsum(M_list)])
    qa, qb, want = _ints(int(off[-1]), off, E, N, K, N + K)
    for t in (torch.bfloat16, torch.float32):
        _check_exact(_product(qa, qb, off, E, N, K, t), want)


# ----------------------------------------------------------- 64-bit offsets

def test_offsets_past_32_bits():
    """2**20 + 77 rows of 4096 dispatched to two rows each: 2**32 source values, more than 2**32 code bytes, and pair
    indices of the requantisation's random words above 2**32; rows at both ends against the oracle."""
    R, C, N = (1 << 20) + 77, 4096, 32
    x = torch.randn((R, C), dtype=torch.bfloat16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    to = torch.arange(2 * R - 1, -1, -1, dtype=torch.int32, device="cuda")        # row r to 2R-1-2r and 2R-2-2r
    codes, sf = m4.mxfp4_quant(x, out_map=to, copies=2)
    rows = np.array([0, 1, R // 2, R - 2, R - 1])
    want = mxfp4.quantize(x[torch.from_numpy(rows).cuda()].float().cpu().numpy())
    del x, to
    for j in (0, 1):
        at = torch.from_numpy(2 * R - 1 - 2 * rows - j).cuda()
        assert_bytes_equal(to_np(codes[at]), want[0], "codes")
        assert_bytes_equal(to_np(sf[at]), want[1], "scales")
    M = 2 * R
    # two experts, the second's rows starting past 2**32 bytes
    off = np.array([0, (1 << 21) + 90, M])
    rng = np.random.default_rng(3)
    bq = rng.integers(0, 256, (2 * N, C // 2), dtype=np.uint8)
    bs = rng.integers(120, 128, (2 * N, C // 32), dtype=np.uint8)
    c = m4.moe_grouped_gemm_mx4(codes, sf, cuda_u8(bq).view(2, N, -1), cuda_u8(bs).view(2, N, -1), cuda_i32(off), torch.float32)
    B = mxfp4.dequant(bq, bs).reshape(2, N, C)
    for i in (0, int(off[1]) - 1, int(off[1]), M - 1):
        A = mxfp4.dequant(to_np(codes[i:i + 1]), to_np(sf[i:i + 1]))
        e = int(i >= off[1])
        # K float32 additions, each off by at most a unit of the terms' magnitude
        assert (np.abs(to_np(c[i:i + 1]) - A @ B[e].T) <= C * 2.0 ** -23 * (np.abs(A) @ np.abs(B[e]).T)).all()
    del c
    offp = mx.padded_offsets(off)
    oc, os_ = m4.mxfp8_requant_mx4_sr_T(codes, sf, cuda_i32(off), cuda_i32(offp), 5, 19, int(offp[-1]))
    r0, r1, P = int(off[1]), M, int(offp[2] - offp[1])
    blk = np.zeros((C, P))
    blk[:, :r1 - r0] = mxfp4.dequant(to_np(codes[r0:r1]), to_np(sf[r0:r1])).T
    e = mx.mx_scale_exponent(np.abs(blk).reshape(C, P // 32, 32).max(axis=2))
    index = (r0 + np.arange(P, dtype=np.uint64))[None, :] * np.uint64(C) + np.arange(C, dtype=np.uint64)[:, None]
    want = mx.round_sr(blk * np.repeat(np.exp2(-e.astype(np.float64)), 32, axis=1), srhash.random16(5, 19, index)).astype(np.uint8)
    a = C * int(offp[1])
    assert_bytes_equal(to_np(os_[a // 32:(a + C * P) // 32]), (e + 127).astype(np.uint8).reshape(-1), "scales")
    assert_bytes_equal(to_np(oc[a:a + C * P]), want.reshape(-1), "codes")
