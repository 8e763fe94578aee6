"""The balance loss and the dense router backward on the GPU against float64:
counts exactly, the rest within the float32 roundings counted at each check;
the layer trained with both, captured and replayed."""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import bf16_from_bits, cuda_f32, cuda_i32, to_np
from oracle import balance as ob
from oracle import formats as fmt
from oracle import route
from oracle import router

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import precision_moe_numerics_quant_amd as m4
    from precision_moe_numerics_quant_amd import layer

U = 2.0 ** -24


def _case(T, E, k, seed, segs=None, masked=0.0, bias=False):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E)).astype(np.float32)
    z[:, 0] += 2.0
    b = (0.5 * rng.standard_normal(E)).astype(np.float32) if bias else None
    idx = route.topk_gates(z, k, b)[0] if T else np.zeros((0, k), np.int32)
    mask = rng.random(T) >= masked if masked else None
    return z, idx, b, mask, segs


def _dev(z, idx, b, mask, segs):
    return (cuda_f32(z), cuda_i32(idx), dict(bias=None if b is None else cuda_f32(b),
                                             token_mask=None if mask is None else torch.from_numpy(mask).cuda(),
                                             seg_off=None if segs is None else cuda_i32(segs)))


def _eps(z, b):
    """Relative error of a float32 softmax: the argument z + b - max rounds twice by at most its magnitude, the
    exponential by two units, the sum of E positive terms at most E / 64 + 6 times on the way through a wave,
    then a reciprocal and a product."""
    y = z + (0 if b is None else b)
    y = np.where(np.isfinite(y), y, np.nan)
    span = float(np.nanmax(np.nanmax(y, 1) - np.nanmin(y, 1))) if y.size else 0.0
    return (2 * span + z.shape[1] / 64 + 6 + 8) * U


CASES = [(1, 2, 1, None, 0, False), (256, 8, 2, None, 0.0, False), (1000, 64, 8, None, 0.3, True), (333, 130, 6, [0, 5, 5, 6, 200, 333], 0.2, True),
         (70, 1024, 16, [0, 70], 0.0, True), (513, 384, 8, [3, 64, 128, 500], 0.0, False), (64, 9, 9, [0] * 5 + [64] * 5, 0.5, False),
         (130, 65, 3, None, 1.0, False), (0, 8, 2, [0, 0, 0], 0.0, False)]


@pytest.mark.parametrize("T,E,k,segs,masked,bias", CASES)
def test_balance_loss_and_gradient(T, E, k, segs, masked, bias):
    c = _case(T, E, k, T + E, segs, masked, bias)
    z, idx, b, mask, _ = c
    lg, ix, kw = _dev(*c)
    r = m4.moe_balance_loss(lg, ix, **kw)
    o = ob.balance_loss(z, idx, b, mask, segs)
    assert np.array_equal(to_np(r["counts"]), o["counts"]) and np.array_equal(to_np(r["tokens"]), o["tokens"])
    eps = _eps(z, b)
    n = max(1, int(o["tokens"].max()))
    tol = eps + (n + 2) * U                                  # a mean of n positive terms
    assert (np.abs(to_np(r["probs"]) - o["probs"]) <= tol * o["probs"]).all()
    tol += (E + 6) * U                                       # then E positive products
    assert (np.abs(to_np(r["loss"]) - o["loss"]) <= tol * o["loss"]).all()
    S = len(o["loss"])
    rng = np.random.default_rng(1)
    dl, base = rng.standard_normal(S).astype(np.float32), (1e-4 * rng.standard_normal((T, E))).astype(np.float32)
    g = ob.balance_grad(dl, z, o["counts"], o["tokens"], k, b, mask, segs)
    got0 = to_np(m4.moe_balance_loss_backward(cuda_f32(dl), lg, r["counts"], r["tokens"], k, **kw)).astype(np.float64)
    got1 = to_np(m4.moe_balance_loss_backward(cuda_f32(dl), lg, r["counts"], r["tokens"], k, dlogits=cuda_f32(base), **kw)).astype(np.float64)
    # f p ((c - m) - sum p (c - m)): the two terms' magnitudes, each with the error of p and a handful of roundings
    lim = np.zeros((T, E))
    for s, (a, e) in enumerate(ob._segments(T, segs)):
        if o["tokens"][s]:
            p = ob.softmax(ob._z(z, b))[a:e]
            cc = np.abs(o["counts"][s] - k * o["tokens"][s] / E)
            f = abs(dl[s]) * E / (k * o["tokens"][s] ** 2)
            lim[a:e] = f * p * (cc + (p @ cc)[:, None]) * (3 * eps + 16 * U)
            # the float64 reference's own roundings: c - p @ c is not centred there, so where the counts are even
            # (exactly 0, which the kernel gives) it leaves E products and sums, each off by 2**-53 of at most max c
            lim[a:e] += f * p * (2 * E + 8) * 2.0 ** -53 * o["counts"][s].max()
    assert (np.abs(got0 - g) <= lim).all()
    assert (np.abs(got1 - (g + base)) <= lim + U * np.abs(g + base) + U * lim).all()


def test_gradient_against_differences():
    z, idx, b, mask, segs = _case(12, 6, 2, 3, [0, 5, 12], 0.2, True)
    lg, ix, kw = _dev(z, idx, b, mask, segs)
    r = m4.moe_balance_loss(lg, ix, **kw)
    w = np.float32([0.7, -1.3])
    g = to_np(m4.moe_balance_loss_backward(cuda_f32(w), lg, r["counts"], r["tokens"], 2, **kw))
    h = 2.0 ** -8
    for t in range(12):
        for e in range(6):
            d = []
            for sgn in (1, -1):
                y = z.copy()
                y[t, e] += np.float32(sgn * h)
                d.append((ob.balance_loss(y, idx, b, mask, segs)["loss"] * w).sum())
            assert abs((d[0] - d[1]) / (2 * h) - g[t, e]) < 4 * h * h * 1.3


def test_masked_tokens_are_not_read():
    """NaN logits and indices far out of range in masked rows, -infinities elsewhere, a row of nothing but
    -infinities: finite everywhere and nothing reported."""
    z, idx, _, _, _ = _case(80, 12, 2, 5)
    mask = np.ones(80, bool)
    mask[[0, 17, 79]] = False
    zz, ii = z.copy(), idx.copy()
    zz[~mask], ii[~mask] = np.nan, 1 << 30
    zz[3, :11] = zz[4] = -np.inf
    lg, ix, kw = _dev(zz, ii, None, mask, [0, 40, 80])
    r = m4.moe_balance_loss(lg, ix, **kw)
    z2 = np.where(np.isnan(zz), 0, zz)
    o = ob.balance_loss(z2, np.where(mask[:, None], idx, 0), None, mask, [0, 40, 80])
    assert np.array_equal(to_np(r["counts"]), o["counts"])
    assert np.allclose(to_np(r["loss"]), o["loss"], rtol=_eps(z, None) + 200 * U)
    base = torch.full((80, 12), 3.0, device="cuda")
    g = m4.moe_balance_loss_backward(torch.ones(2, device="cuda"), lg, r["counts"], r["tokens"], 2, dlogits=base, **kw)
    assert torch.isfinite(g).all() and (g[~torch.from_numpy(mask).cuda()] == 3.0).all() and (g[4] == 3.0).all()
    m4.moe4_debug_check()
    ix[5, 0] = 12
    m4.moe_balance_loss(lg, ix, **kw)
    with pytest.raises(m4.Moe4DeviceError, match="clamped"):
        m4.moe4_debug_check()


def test_balance_deterministic_in_place_and_replayed():
    c = _case(2000, 384, 8, 9, [0, 700, 2000], 0.1, True)
    lg, ix, kw = _dev(*c)
    base = torch.randn((2000, 384), device="cuda") * 1e-5
    dl = torch.ones(2, device="cuda")

    def step(dz):
        r = m4.moe_balance_loss(lg, ix, **kw)
        m4.moe_balance_loss_backward(dl, lg, r["counts"], r["tokens"], 8, dlogits=dz, out=dz, **kw)
        return r["loss"], r["probs"], dz
    ref = [t.clone() for t in step(base.clone())]
    out = m4.moe_balance_loss_backward(dl, lg, m4.moe_balance_loss(lg, ix, **kw)["counts"], m4.moe_balance_loss(lg, ix, **kw)["tokens"], 8,
                                       dlogits=base, **kw)
    assert torch.equal(out, ref[2])
    buf = base.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(base.clone())
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        buf.copy_(base)
        outs = step(buf)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
        step(base.clone())
        torch.cuda.synchronize()


def test_two_calls_at_once():
    """Calls in flight on two streams (each with its own workspace) give the bits of calls made alone."""
    rng = np.random.default_rng(21)
    cases = []
    for T, E, d in ((4000, 384, 516), (3000, 64, 260)):
        z = cuda_f32(rng.standard_normal((T, E)).astype(np.float32))
        idx = cuda_i32(rng.integers(0, E, (T, 4)).astype(np.int32))
        off = cuda_i32(np.array([0, 7, 7, T // 2, T], np.int32))
        x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda().bfloat16()

        def step(z=z, idx=idx, off=off, x=x):
            b = m4.moe_balance_loss(z, idx, seg_off=off)
            dz = m4.moe_balance_loss_backward(torch.ones(4, device="cuda"), z, b["counts"], b["tokens"], 4, seg_off=off)
            return [b["loss"], b["counts"], dz, m4.moe_router_wgrad_dense(x, dz)]
        cases.append(step)
    alone = [[v.cpu() for v in step()] for step in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(4):
        for i, (step, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i].append(step())
    torch.cuda.synchronize()
    for want, runs in zip(alone, got):
        for run in runs:
            assert all(torch.equal(w, v.cpu()) for w, v in zip(want, run))


# -------------------------------------------------------------- dense router

@pytest.mark.parametrize("T,E,k,d", [(1, 2, 1, 4), (200, 8, 2, 256), (333, 130, 6, 520), (50, 20, 16, 68), (130, 384, 8, 1024), (2500, 33, 3, 132),
                                     (129, 129, 1, 132), (4100, 70, 3, 1028)])
def test_dense_router_backward(T, E, k, d):
    rng = np.random.default_rng(T + d)
    inv = rng.permutation(T * k).astype(np.int32)
    dxp = (1e-2 * rng.standard_normal((T * k, d))).astype(np.float32)
    dz = (rng.standard_normal((T, E)) * np.exp2(rng.integers(-12, 1, (T, E)))).astype(np.float32)
    xb, wb = fmt.f64_to_bf16(rng.standard_normal((T, d))), fmt.f64_to_bf16(0.05 * rng.standard_normal((E, d)))
    dx = m4.moe_unpermute_sum_router_dense(cuda_f32(dxp), cuda_i32(inv), T, k, cuda_f32(dz), bf16_from_bits(wb))
    exact, mag = router.unpermute_sum_dense(dxp, inv, T, k, dz, wb)
    # exact products; k + 3 E additions of float32 (three parts of each dz), cut or rounded, then half a bf16 unit
    slack = (k + 3 * E + 2) * 2 * U * mag
    lim = slack + 2.0 ** -8 * np.exp2(np.floor(np.log2(np.abs(exact) + slack + 1e-300)))
    assert (np.abs(dx.float().cpu().numpy() - exact) <= lim).all()
    dw = to_np(m4.moe_router_wgrad_dense(bf16_from_bits(xb), cuda_f32(dz)))
    exact, mag = router.weight_grad_dense(xb, dz)
    assert (np.abs(dw - exact) <= (3 * T + 8) * 2 * U * mag).all()
    again = to_np(m4.moe_router_wgrad_dense(bf16_from_bits(xb), cuda_f32(dz)))
    assert np.array_equal(dw.view(np.uint32), again.view(np.uint32))
    m4.moe4_debug_check()


def test_dense_router_split_is_exact():
    """One-hot operands: each result is one product dz * w (or dz * x) with dz of 24 significant bits and a power
    of two, which only the exact three-part split reproduces."""
    rng = np.random.default_rng(7)
    T = E = 64
    d = 64
    dz = (rng.integers(1 << 23, 1 << 24, (T, E)).astype(np.float64) * np.exp2(rng.integers(-60, -20, (T, E)))).astype(np.float32)
    dz *= np.where(rng.random((T, E)) < 0.5, -1, 1).astype(np.float32)
    eye = fmt.f64_to_bf16(np.eye(64) * 0.5)
    dw = to_np(m4.moe_router_wgrad_dense(bf16_from_bits(eye), cuda_f32(dz)))       # dw[e, c] = dz[c, e] / 2
    assert np.array_equal(dw, dz.T * np.float32(0.5))


def test_dense_router_gradients_that_are_not_finite():
    """A NaN (every mantissa bit set) and an infinity spoil their token's dx and their expert's dW, and nothing else."""
    T, E, d, k = 130, 40, 64, 2
    rng = np.random.default_rng(3)
    dz = rng.standard_normal((T, E)).astype(np.float32)
    dz.view(np.uint32)[3, 5] = 0x7FFFFFFF
    dz[129, 39] = np.inf
    w = fmt.f64_to_bf16(1 + rng.random((E, d)))
    x = fmt.f64_to_bf16(1 + rng.random((T, d)))
    dx = m4.moe_unpermute_sum_router_dense(cuda_f32(np.ones((T * k, d), np.float32)), cuda_i32(rng.permutation(T * k).astype(np.int32)),
                                           T, k, cuda_f32(dz), bf16_from_bits(w)).float().cpu().numpy()
    bad = np.isin(np.arange(T), [3, 129])
    assert not np.isfinite(dx[bad]).any() and np.isfinite(dx[~bad]).all()
    dw = to_np(m4.moe_router_wgrad_dense(bf16_from_bits(x), cuda_f32(dz)))
    bad = np.isin(np.arange(E), [5, 39])
    assert not np.isfinite(dw[bad]).any() and np.isfinite(dw[~bad]).all()


def test_dense_router_empty_batch_and_bad_rows():
    w = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    dw = m4.moe_router_wgrad_dense(x, torch.zeros((0, 8), device="cuda"))
    assert dw.shape == (8, 64) and not dw.any()
    dx = m4.moe_unpermute_sum_router_dense(torch.ones((2, 64), device="cuda"), cuda_i32([5, -1]), 2, 1, torch.zeros((2, 8), device="cuda"), w)
    assert (dx == 1).all()
    with pytest.raises(m4.Moe4DeviceError, match="clamped"):
        m4.moe4_debug_check()


@pytest.mark.parametrize("variant", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("side", [False, True])
def test_layer_with_balance_and_router(variant, side, monkeypatch):
    """The tiny layer with its router and the balance loss: dlogits = the routed gradient + the balance gradient,
    dx and dW_router from the dense logit gradient; a graph of the step replays to the eager step's results."""
    if side:
        monkeypatch.setattr(layer, "SIDE_STREAM_MIN_ELEMS", 0)
    inp = synth.config_inputs(1, device="cpu")
    c = synth.CONFIGS[1]
    T, d, E, k = c["T"], c["d"], c["E"], c["k"]
    wb = fmt.f64_to_bf16(0.05 * np.random.default_rng(11).standard_normal((E, d)))
    dev = {n: (v.cuda() if torch.is_tensor(v) else v) for n, v in inp.items()}
    rw, seg = bf16_from_bits(wb), [0, 100, 100, 256]
    mask = np.ones(T, bool)
    mask[90:100] = False
    mk, so, coef = torch.from_numpy(mask).cuda(), cuda_i32(seg), cuda_f32([0.01, 0.01, 0.02])
    f, b = (layer.forward, layer.backward) if variant == "nvfp4" else (layer.forward_mx4, layer.backward_mx4)

    def step(dbal=coef):
        fw = f(dev["x"], dev["w_up"], dev["w_down"], None, k, seed=synth.SR_SEED, router_w=rw, balance=True, token_mask=mk, seg_off=so)
        return fw, b(fw, dev["dy"], seed=synth.SR_SEED, dbalance=dbal)
    fw, bw = step()
    plain = b(fw, dev["dy"], seed=synth.SR_SEED)
    lg, idx = to_np(fw["logits"]), to_np(fw["route"]["idx"])
    o = ob.balance_loss(lg, idx, None, mask, seg)
    assert np.array_equal(to_np(fw["balance"]["counts"]), o["counts"])
    g = ob.balance_grad(to_np(coef), lg, o["counts"], o["tokens"], k, None, mask, seg)
    dl, routed = to_np(bw["dlogits"]).astype(np.float64), to_np(plain["dlogits"]).astype(np.float64)
    assert (np.abs(dl - (routed + g)) <= 1e-5 * np.abs(g).max() + 2 * U * np.abs(routed)).all() and np.abs(g).max() > 0
    exact, mag = router.unpermute_sum_dense(to_np(bw["dXp"]), to_np(fw["route"]["inv_perm"]), T, k, to_np(bw["dlogits"]), wb)
    slack = (k + 3 * E + 2) * 2 * U * mag
    lim = slack + 2.0 ** -8 * np.exp2(np.floor(np.log2(np.abs(exact) + slack + 1e-300)))
    assert (np.abs(bw["dx"].float().cpu().numpy() - exact) <= lim).all()
    exact, mag = router.weight_grad_dense(synth.bf16_bits(inp["x"]), to_np(bw["dlogits"]))
    assert (np.abs(to_np(bw["dW_router"]) - exact) <= (3 * T + 8) * 2 * U * mag).all()
    outs = lambda fw, bw: [fw["y"], fw["balance"]["loss"], bw["dx"], bw["dlogits"], bw["dW_router"], bw["dW_up"]]
    ref = [t.clone() for t in outs(fw, bw)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = outs(*step())
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        step()
        torch.cuda.synchronize()
    with pytest.raises(ValueError, match="balance=True"):
        b({n: v for n, v in fw.items() if n != "balance"}, dev["dy"], dbalance=coef)
