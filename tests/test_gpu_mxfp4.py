"""MXFP4 on the GPU against the oracle: codes, scales, decode and the
transposed requantisation byte for byte; the grouped product per element; the
layer with the MXFP4 forward, teacher-forced, captured and replayed."""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import assert_bytes_equal, bf16_from_bits, cuda_f32, cuda_i32, cuda_u8, to_np
from oracle import formats as fmt
from oracle import gemm as og
from oracle import layer as olayer
from oracle import mxfp4
from oracle import mxfp8 as mx
from oracle import nvfp4 as nv
from oracle import route
from oracle import silu as osilu

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import precision_moe_numerics_quant_amd as m4
    from precision_moe_numerics_quant_amd import layer

LAYOUTS = {0: mx.SF_ROWS, 1: mx.SF_BLOCKS}


def _x(R, C, seed):
    return synth.activations(R, C, "cpu", seed, outlier_p=0.002, outlier_mul=30.0)


def _check(got, want, what):
    assert_bytes_equal(to_np(got[1]), want[1], what + " scales")
    assert_bytes_equal(to_np(got[0]), want[0], what + " codes")


# --------------------------------------------------------------------- quant

@pytest.mark.parametrize("R,C", [(1, 32), (1, 4096), (3, 64), (77, 544), (333, 1536)])
def test_quant_bf16_and_f32(R, C):
    x = _x(R, C, R + C)
    _check(m4.mxfp4_quant(x.cuda()), mxfp4.quantize(x.float().numpy()), "bf16")
    w = synth.randn((R, C), 0.02, "cpu", R, "w_up")
    w[:, ::7] *= torch.exp2(torch.randint(-60, 60, (R, 1)).float())
    _check(m4.mxfp4_quant(w.cuda()), mxfp4.quantize(w.numpy()), "f32")


def test_quant_special_blocks():
    """Zeros of both signs, infinities, NaN, the largest and smallest numbers, exact ties, and blocks whose
    amax sits at and next to the scale rule's borders."""
    f = np.finfo(np.float32)
    x = np.ones((1, 32 * 16), np.float32)
    b = x.reshape(16, 32)
    b[0, 3], b[1, 5], b[2, 31] = np.inf, np.nan, -np.inf
    b[3], b[4] = 0.0, -0.0
    b[5, 0], b[6], b[7, 0] = f.max, f.smallest_subnormal, -f.tiny
    b[8, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25]
    b[9, 0], b[10, 0], b[11, 0] = 6.0, np.nextafter(np.float32(6), np.float32(7)), np.nextafter(np.float32(6), np.float32(5))
    b[12] = np.float32(2.0 ** -126) * np.arange(32, dtype=np.float32)
    b[13, 0], b[14] = 2.0 ** 127, 2.0 ** -130
    want = mxfp4.quantize(x)
    got = m4.mxfp4_quant(cuda_f32(x))
    _check(got, want, "special")
    for dt in (torch.float32, torch.bfloat16):
        v = m4.mxfp4_dequant(*got, dt).float().cpu().numpy()
        ref = mxfp4.dequant(*want)
        with np.errstate(over="ignore"):
            assert np.array_equal(v, ref.astype(np.float32), equal_nan=True)     # (2**128 is an infinity)
        assert np.array_equal(np.signbit(v)[~np.isnan(v)], np.signbit(ref)[~np.isnan(v)])


def test_quant_silu_every_bf16_pattern():
    """silu of all finite bf16 patterns, and of the infinities and NaN: +inf and NaN blocks are NaN, silu(-inf) is -0."""
    bits = np.arange(65536, dtype=np.uint16)
    fin = bits[(bits & 0x7F80) != 0x7F80]
    fin = np.concatenate([fin, np.zeros((-len(fin)) % 2048, np.uint16)]).reshape(-1, 2048)
    _check(m4.mxfp4_quant(bf16_from_bits(fin), m4.PRE_SILU), mxfp4.quantize(osilu.silu_f32(fin)), "silu")
    x = np.full((1, 128), 0x3F80, np.uint16)
    x[0, 0], x[0, 32], x[0, 64] = 0x7F80, 0x7FC0, 0xFF80
    codes, sf = m4.mxfp4_quant(bf16_from_bits(x), m4.PRE_SILU)
    assert to_np(sf)[0].tolist() == [255, 255, 124, 124]     # silu(1) = 0.731 = 5.85 * 2**-3
    assert nv.unpack_codes(to_np(codes))[0, 64] == 8


@pytest.mark.parametrize("R,C,copies", [(1, 32, 1), (5, 1056, 8), (200, 64, 3), (129, 4096, 8)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quant_dispatch(R, C, copies, dt):
    """Each row to its named output rows; rows that no entry names keep what they held."""
    x = _x(R, C, R).float() if dt == "f32" else _x(R, C, R)
    q, s = mxfp4.quantize(x.float().numpy())
    rng = np.random.default_rng(R)
    n_out = R * copies + 5
    to = rng.permutation(n_out)[:R * copies]
    out = (torch.full((n_out, C // 2), 0xA5, dtype=torch.uint8, device="cuda"),
           torch.full((n_out, C // 32), 0x5A, dtype=torch.uint8, device="cuda"))
    got = m4.mxfp4_quant(x.cuda(), out_map=cuda_i32(to), copies=copies, out=out)
    wq, ws = np.full((n_out, C // 2), 0xA5, np.uint8), np.full((n_out, C // 32), 0x5A, np.uint8)
    wq[to], ws[to] = np.repeat(q, copies, 0), np.repeat(s, copies, 0)
    _check(got, (wq, ws), "dispatch")
    m4.moe4_debug_check()


def test_quant_dispatch_reports_rows_outside():
    x = _x(4, 64, 1)
    codes, sf = m4.mxfp4_quant(x.cuda(), out_map=cuda_i32([0, -1, 4, 2]), copies=1)
    with pytest.raises(m4.Moe4DeviceError, match="clamped"):
        m4.moe4_debug_check()
    q, s = mxfp4.quantize(x.float().numpy())
    assert np.array_equal(to_np(codes)[[0, 2]], q[[0, 3]]) and np.array_equal(to_np(sf)[[0, 2]], s[[0, 3]])
    m4.moe4_debug_check()


def test_dequant_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))[:, :256].reshape(256, 256)
    sf = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    ref = mxfp4.dequant(codes, sf)
    with np.errstate(over="ignore"):
        ref = ref.astype(np.float32)
    for dt in (torch.float32, torch.bfloat16):
        v = m4.mxfp4_dequant(cuda_u8(codes), cuda_u8(sf), dt)
        assert np.array_equal(v.float().cpu().numpy(), ref, equal_nan=True)


# ------------------------------------------------------------------- requant

@pytest.mark.parametrize("lay", [0, 1])
@pytest.mark.parametrize("sizes,C", [([1], 32), ([31, 0, 33, 0, 1], 544), ([0, 0], 64), ([130, 64, 7], 1056), ([32, 96], 512)])
def test_requant_bit_exact(sizes, C, lay):
    off = np.concatenate([[0], np.cumsum(sizes)])
    offp = mx.padded_offsets(off)
    R, P = int(off[-1]), int(offp[-1])
    q, s = mxfp4.quantize(_x(max(R, 1), C, C).float().numpy()[:R] if R else np.zeros((0, C), np.float32))
    oc, os_ = m4.mxfp8_requant_mx4_sr_T(cuda_u8(q), cuda_u8(s), cuda_i32(off), cuda_i32(offp), 5, 19, P, lay)
    wc, ws = mxfp4.requant_sr_t(q, s, off, 5, 19, LAYOUTS[lay])
    assert_bytes_equal(to_np(os_), ws, "scales")
    assert_bytes_equal(to_np(oc), wc, "codes")


def test_requant_scales_at_the_ends():
    """Scale bytes 0 .. 9 and 240 .. 254 (subnormal and near-overflow values), and bytes of 255: those columns' blocks get 255."""
    rng = np.random.default_rng(4)
    q = rng.integers(0, 256, (64, 64), dtype=np.uint8)
    for lo, hi in ((0, 10), (240, 254)):
        s = rng.integers(lo, hi, (64, 4), dtype=np.uint8)
        off = [0, 64]
        got = m4.mxfp8_requant_mx4_sr_T(cuda_u8(q), cuda_u8(s), cuda_i32(off), cuda_i32(off), 1, 2, 64)
        want = mxfp4.requant_sr_t(q, s, off, 1, 2)
        _check(got, want, "ends")
    s = np.full((64, 4), 127, np.uint8)
    s[3, 1] = 255
    _, os_ = m4.mxfp8_requant_mx4_sr_T(cuda_u8(q), cuda_u8(s), cuda_i32(off), cuda_i32(off), 1, 2, 64)
    b = to_np(os_).reshape(128, 2)
    assert (b[32:64, 0] == 255).all() and (b[32:64, 1] != 255).all() and (b[:32] != 255).all() and (b[64:] != 255).all()


# ------------------------------------------------------------------- product

def _gemm_check(got, exact, bound, K, bf16):
    """Products are exact; a float32 accumulation of K terms rounds at most K times, each by at most one unit
    (2**-23, a cut as well as a rounding) of a partial sum that is at most the terms' magnitude; then one
    rounding to the output type, half a unit of it."""
    slack = K * 2.0 ** -23 * bound
    a = np.maximum(np.abs(exact) + slack, 2.0 ** -126)
    lim = slack + 0.5 * np.exp2(np.floor(np.log2(a)) - (7 if bf16 else 23))
    err = np.abs(got - exact)
    assert (err <= lim).all(), float((err / lim).max())


def _operands(M_list, N, K, seed):
    E = len(M_list)
    off = np.concatenate([[0], np.cumsum(M_list)]).astype(np.int64)
    qa = mxfp4.quantize(_x(max(int(off[-1]), 1), K, seed).float().numpy()[:int(off[-1])])
    qb = mxfp4.quantize(synth.randn((E * N, K), 0.02, "cpu", seed, "w_up").numpy())
    return off, qa, qb


def _product(off, qa, qb, N, K, dt):
    E = len(off) - 1
    return m4.moe_grouped_gemm_mx4(cuda_u8(qa[0]), cuda_u8(qa[1]), cuda_u8(qb[0]).view(E, N, K // 2),
                                   cuda_u8(qb[1]).view(E, N, K // 32), cuda_i32(off), dt)


# many and few rows per expert, K with and without whole 128- and 256-value
# steps, N with and without whole 128- and 256-row tiles, empty experts
GEMMS = [([1], 32, 32), ([0, 0, 1, 0], 64, 96), ([3, 0, 17, 1, 33], 96, 160), ([5, 300, 0, 129], 160, 256), ([256], 128, 256),
         ([0, 37, 130, 1, 300], 256, 384), ([0, 37, 130, 1, 300], 384, 512), ([2100, 700, 1, 0, 900], 1280, 256),
         ([700, 1500, 3], 1024, 544), ([0, 1, 2, 3, 5, 9, 10, 13, 16, 17, 31, 32, 33, 70, 0, 4, 8, 12], 192, 1536),
         ([1, 0, 0, 1, 1, 0, 1], 1536, 4096), ([200, 0, 90], 32, 64)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M_list,N,K", GEMMS)
def test_gemm(M_list, N, K, dt):
    off, qa, qb = _operands(M_list, N, K, N + K)
    got = _product(off, qa, qb, N, K, torch.bfloat16 if dt == "bf16" else torch.float32).float().cpu().numpy().astype(np.float64)
    A, B = mxfp4.dequant(*qa), mxfp4.dequant(*qb).reshape(len(M_list), N, K)
    _gemm_check(got, og.grouped_nt(A, B, off), og.abs_bound_nt(A, B, off), K, dt == "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(288, 512), (288, 160), (544, 512)])
def test_gemm_many_experts_of_few_rows(N, K, dt):
    """Between the few-rows kernel's four rows per expert and a tile's 128: most experts end inside a tile."""
    M_list = [(7 * i) % 23 if i % 3 else 0 for i in range(159)] + [301]
    off, qa, qb = _operands(M_list, N, K, N + K)
    got = _product(off, qa, qb, N, K, torch.bfloat16 if dt == "bf16" else torch.float32).float().cpu().numpy().astype(np.float64)
    A, B = mxfp4.dequant(*qa), mxfp4.dequant(*qb).reshape(len(M_list), N, K)
    _gemm_check(got, og.grouped_nt(A, B, off), og.abs_bound_nt(A, B, off), K, dt == "bf16")


@pytest.mark.parametrize("shift_a,shift_b", [(1, 0), (0, 3), (2, 1)])
@pytest.mark.parametrize("M_list,N,K", [([150, 3, 77], 160, 512), ([2, 1], 64, 512), ([90, 40], 96, 544)])
def test_gemm_scales_at_any_alignment(M_list, N, K, shift_a, shift_b):
    """Scale tensors that start at any byte (a view into a larger buffer)."""
    off, qa, qb = _operands(M_list, N, K, 5)
    E = len(M_list)

    def at(s, n):
        buf = torch.empty(s.size + 16, dtype=torch.uint8, device="cuda")
        v = buf[n:n + s.size].view(s.shape)
        v.copy_(torch.from_numpy(s))
        return v
    want = _product(off, qa, qb, N, K, torch.float32)
    got = m4.moe_grouped_gemm_mx4(cuda_u8(qa[0]), at(qa[1], shift_a), cuda_u8(qb[0]).view(E, N, K // 2),
                                  at(qb[1], shift_b).view(E, N, K // 32), cuda_i32(off), torch.float32)
    assert torch.equal(got, want)


@pytest.mark.parametrize("M_list,N,K", [([50, 0, 90], 64, 128), ([300, 200], 256, 512), ([7, 0, 20, 3], 128, 96)])
def test_gemm_exact_small_integers(M_list, N, K):
    """Small values under scales near one: every partial sum is exact in float32."""
    rng = np.random.default_rng(3)
    off = np.concatenate([[0], np.cumsum(M_list)])
    a, b = rng.integers(0, 256, (off[-1], K // 2), dtype=np.uint8), rng.integers(0, 256, (len(M_list) * N, K // 2), dtype=np.uint8)
    sa = rng.integers(125, 130, (off[-1], K // 32), dtype=np.uint8)
    sb = rng.integers(125, 130, (len(M_list) * N, K // 32), dtype=np.uint8)
    got = to_np(_product(off, (a, sa), (b, sb), N, K, torch.float32)).astype(np.float64)
    assert np.array_equal(got, og.grouped_nt(mxfp4.dequant(a, sa), mxfp4.dequant(b, sb).reshape(len(M_list), N, K), off))


@pytest.mark.parametrize("M_list,N,K", [([3, 1], 64, 256), ([150, 200], 128, 512)])
def test_gemm_scales_at_the_ends_and_nan(M_list, N, K):
    """Scale bytes whose products reach the smallest and largest float32 normals; a scale byte of 255 makes its row or column NaN."""
    rng = np.random.default_rng(5)
    off = np.concatenate([[0], np.cumsum(M_list)])
    E, M = len(M_list), int(off[-1])
    a, b = rng.integers(0, 256, (M, K // 2), dtype=np.uint8), rng.integers(0, 256, (E * N, K // 2), dtype=np.uint8)
    for ea, eb in ((60, 80), (180, 170), (1, 250)):
        sa, sb = np.full((M, K // 32), ea, np.uint8), np.full((E * N, K // 32), eb, np.uint8)
        got = to_np(_product(off, (a, sa), (b, sb), N, K, torch.float32)).astype(np.float64)
        A, B = mxfp4.dequant(a, sa), mxfp4.dequant(b, sb).reshape(E, N, K)
        _gemm_check(got, og.grouped_nt(A, B, off), og.abs_bound_nt(A, B, off), K, False)
    sa, sb = np.full((M, K // 32), 127, np.uint8), np.full((E * N, K // 32), 127, np.uint8)
    sa[1, 2], sb[N + 5, 0] = 255, 255
    got = to_np(_product(off, (a, sa), (b, sb), N, K, torch.float32))
    nan = np.zeros((M, N), bool)
    nan[1], nan[off[1]:, 5] = True, True
    assert np.array_equal(np.isnan(got), nan)


def test_gemm_leaves_other_rows_alone_and_is_deterministic():
    """Rows of C behind the last expert's are not written (through the C call, C pre-filled)."""
    import ctypes
    off, qa, qb = _operands([40, 0, 23], 96, 160, 1)
    E, N, K, M = 3, 96, 160, 70
    qa = tuple(np.concatenate([q, np.full((7, q.shape[1]), 0xFF, np.uint8)]) for q in qa)
    a, s, b, t, o = cuda_u8(qa[0]), cuda_u8(qa[1]), cuda_u8(qb[0]), cuda_u8(qb[1]), cuda_i32(off)
    outs = []
    for _ in range(2):
        c = torch.full((M, N), 7.0, device="cuda")
        rc = m4.lib().moe_grouped_gemm_mx4(*(ctypes.c_void_p(x.data_ptr()) for x in (a, s, b, t, o)), E, M, N, K,
                                           ctypes.c_void_p(c.data_ptr()), m4.F32, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert rc == 0
        outs.append(c)
    assert torch.equal(outs[0], outs[1]) and (outs[0][63:] == 7.0).all() and torch.isfinite(outs[0][:63]).all()


# ----------------------------------------------------------------- the layer

def _tiny():
    inp = synth.config_inputs(1, device="cpu")
    return inp, synth.CONFIGS[1], {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in inp.items()}


def test_layer_mx4_teacher_forced():
    inp, c, dev = _tiny()
    T, d, F, E, k = c["T"], c["d"], c["F"], c["E"], c["k"]
    fw = layer.forward_mx4(dev["x"], dev["w_up"], dev["w_down"], dev["logits"], k, seed=synth.SR_SEED)
    bw = layer.backward_mx4(fw, dev["dy"], seed=synth.SR_SEED)
    torch.cuda.synchronize()
    o = olayer.forward_mx4(synth.bf16_bits(inp["x"]), inp["w_up"].numpy(), inp["w_down"].numpy(), inp["logits"].numpy(), k)
    P = o["perm"]
    _check(fw["xq_perm"], (o["xq_perm"]["codes"], o["xq_perm"]["sf"]), "X")
    for n, w in (("wu", o["wu"]), ("wd", o["wd"])):
        _check(fw["wq"][n], (w["codes"], w["sf"]), n)
    A, B = mxfp4.dequant(o["xq_perm"]["codes"], o["xq_perm"]["sf"]), mxfp4.dequant(o["wu"]["codes"], o["wu"]["sf"]).reshape(E, F, d)
    U = to_np(fw["U"])
    _gemm_check(fmt.bf16_to_f32(U).astype(np.float64), og.grouped_nt(A, B, P["off"]), og.abs_bound_nt(A, B, P["off"]), d, True)
    hq = mxfp4.quantize(osilu.silu_f32(U))                   # from the GPU's U
    _check(fw["hq"], hq, "H")
    A, B = mxfp4.dequant(*hq), mxfp4.dequant(o["wd"]["codes"], o["wd"]["sf"]).reshape(E, d, F)
    Yp = to_np(fw["Yp"])
    _gemm_check(Yp.astype(np.float64), og.grouped_nt(A, B, P["off"]), og.abs_bound_nt(A, B, P["off"]), F, False)
    assert_bytes_equal(to_np(fw["y"]), olayer.combine(Yp, o["gates"], P["inv_perm"], k), "y")
    # the backward's requantised operands, each from the operand that the GPU made
    for name, q, goff, role, lay in (("wdT", o["wd"], np.arange(E + 1) * d, 3, 0), ("wuT", o["wu"], np.arange(E + 1) * F, 2, 0),
                                     ("hT", dict(codes=hq[0], sf=hq[1]), P["off"], 1, 1), ("xT", o["xq_perm"], P["off"], 0, 1)):
        want = mxfp4.requant_sr_t(q["codes"], q["sf"], goff, synth.SR_SEED, role, LAYOUTS[lay])
        n = len(want[0])
        assert_bytes_equal(to_np(bw[name][1])[:len(want[1])], want[1], name + " scales")
        assert_bytes_equal(to_np(bw[name][0])[:n], want[0], name + " codes")
    dXp = to_np(bw["dXp"])
    assert_bytes_equal(to_np(bw["dx"]), olayer.unpermute_sum(dXp, P["inv_perm"], T, k), "dx")
    for n in ("dW_up", "dW_down", "dg", "dlogits"):
        assert torch.isfinite(bw[n]).all()


def test_layer_mx4_serving_one_token():
    """One token through the layer with weights laid out once (no masters, no backward copies) equals the same
    token in a batch: every step treats rows alone."""
    inp, c, dev = _tiny()
    wq = layer.quantize_weights_mx4(dev["w_up"], dev["w_down"], backward=False)
    all_y = layer.forward_mx4(dev["x"], None, None, dev["logits"], c["k"], wq=wq)["y"]
    for t in (0, 100, 255):
        y = layer.forward_mx4(dev["x"][t:t + 1], None, None, dev["logits"][t:t + 1].contiguous(), c["k"], wq=wq)["y"]
        # the two may take different kernels, whose float32 sums differ in order: bf16 neighbours at the most
        a, b = y.float(), all_y[t:t + 1].float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs().clamp(min=float(b.abs().mean()))).all()
    # the requantisations that the serving copy left out are made by the backward
    fw = layer.forward_mx4(dev["x"], None, None, dev["logits"], c["k"], wq=wq)
    full = layer.forward_mx4(dev["x"], dev["w_up"], dev["w_down"], dev["logits"], c["k"])
    a, b = layer.backward_mx4(fw, dev["dy"]), layer.backward_mx4(full, dev["dy"])
    for n in ("dx", "dW_up", "dW_down", "dlogits"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("T", [1, 256])
def test_layer_mx4_graph_replay(T):
    inp, c, dev = _tiny()
    wq = layer.quantize_weights_mx4(dev["w_up"], dev["w_down"])
    x, lg, dy = (dev[n][:T].contiguous() for n in ("x", "logits", "dy"))

    def step():
        fw = layer.forward_mx4(x, None, None, lg, c["k"], wq=wq)
        bw = layer.backward_mx4(fw, dy)
        return [fw["y"], bw["dx"], bw["dW_up"], bw["dW_down"], bw["dlogits"]]
    ref = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, ref):
            assert torch.equal(a, b)
        step()
        torch.cuda.synchronize()


def test_gemm_full_size_sampled():
    """The training shape (131072 skewed rows, 384 experts, N = 1536, K = 4096) and the rollout shape (4096 rows)
    on sampled rows."""
    for T, zipf in ((16384, 1.1), (512, 0.0)):
        E, k, N, K = 384, 8, 1536, 4096
        lg = synth.randn((T, E), 1.0, "cuda", 0, "logits") + (synth.zipf_bias(E, zipf, "cuda") if zipf else 0)
        r = m4.moe_route_topk(lg.contiguous(), k)
        x = synth.activations(T, K, "cuda", 1)
        a = m4.mxfp4_quant(x, out_map=r["inv_perm"], copies=k)
        w = synth.randn((E * N, K), 0.02, "cuda", 2, "w_up")
        b = m4.mxfp4_quant(w)
        del w
        c = m4.moe_grouped_gemm_mx4(*a, b[0].view(E, N, -1), b[1].view(E, N, -1), r["off"], torch.float32)
        off = to_np(r["off"])
        rows = np.unique(np.linspace(0, T * k - 1, 24).astype(int))
        for i in rows:
            e = int(np.searchsorted(off, i, side="right") - 1)
            A = mxfp4.dequant(to_np(a[0][i:i + 1]), to_np(a[1][i:i + 1]))
            B = mxfp4.dequant(to_np(b[0][e * N:(e + 1) * N]), to_np(b[1][e * N:(e + 1) * N]))
            _gemm_check(to_np(c[i:i + 1]).astype(np.float64), A @ B.T, np.abs(A) @ np.abs(B).T, K, False)
