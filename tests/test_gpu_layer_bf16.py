"""The BF16 layer on the GPU: forward and backward, gated and plain, with
biases, a shared expert, residual, dropout, the router and its balance loss,
against the float64 oracle on the GPU's own routing."""
import numpy as np
import pytest
import torch

import synth
from bf16_helpers import bf
from gpu_helpers import to_np
from oracle import bf16 as ob

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import precision_moe_numerics_quant_amd as m4
    from precision_moe_numerics_quant_amd import layer

T, D, F, E, K = 70, 72, 40, 6, 3


def _weights(rng, gated, e):
    w = {}
    w["w_up"] = bf(rng.standard_normal((e, 2, F, D) if gated else (e, F, D)) * 0.3)
    w["w_down"] = bf(rng.standard_normal((e, D, F)) * 0.3)
    b = [rng.standard_normal(s).astype(np.float32) * 0.5 for s in (w["w_up"][0].shape[:-1], (e, D))]
    w["b_up"], w["b_down"] = [(v.astype(np.float64), torch.from_numpy(v)) for v in b]
    return w


def _gpu(w):
    return {n: v[1].cuda() for n, v in w.items()}


def _block(x, w, act, gated):
    """The forward of one expert's block in float64 and the gradient function."""
    z = x @ w["w_up"].reshape(-1, D).T + w["b_up"].reshape(-1)
    f, df = ob.act(act, z[:, :F])
    h = f * z[:, F:] if gated else f
    y = h @ w["w_down"].T + w["b_down"]

    def grad(dy):
        dh = dy @ w["w_down"]
        dz = np.concatenate([dh * z[:, F:] * df, dh * f], 1) if gated else dh * df
        return dict(dx=dz @ w["w_up"].reshape(-1, D), dW_up=dz.T @ x, db_up=dz.sum(0), dW_down=dy.T @ h, db_down=dy.sum(0))
    return y, grad


def _reference(x, dy, w, sh, r, act, gated, residual, p, seed):
    """y and every gradient of sum(dy * y), the routing given."""
    off, perm, inv, gates = (to_np(r[n]).astype(np.int64) if n != "gates" else to_np(r[n]).astype(np.float64)
                             for n in ("off", "perm", "inv_perm", "gates"))
    keep, fac = ob.keep_mask(T, D, p, seed, 4)
    dyd = np.where(keep, dy * fac, 0.0)
    yp = np.zeros((T * K, D))
    g = dict(dW_up=np.zeros((E,) + w["w_up"].shape[1:]), dW_down=np.zeros((E, D, F)), db_up=np.zeros((E,) + w["b_up"].shape[1:]),
             db_down=np.zeros((E, D)), dx=np.zeros((T, D)), dg=np.zeros(T * K))
    for e, a, b in ob.groups(off):
        rows = perm[a:b]
        y, grad = _block(x[rows // K], {n: v[e] for n, v in w.items()}, act, gated)
        yp[a:b] = y
        gr = grad(gates.reshape(-1)[rows, None] * dyd[rows // K])
        for n in ("dW_up", "dW_down", "db_up", "db_down"):
            g[n][e] = gr[n].reshape(g[n][e].shape)
        np.add.at(g["dx"], rows // K, gr["dx"])
        g["dg"][rows] = (dyd[rows // K] * y).sum(1)
    acc = (gates[:, :, None] * yp[inv.reshape(T, K)]).sum(1)
    out = np.where(keep, acc * fac, 0.0) + (0 if residual is None else residual)
    if sh is not None:
        y, grad = _block(x, {n: v[0] for n, v in sh.items()}, act, gated)
        out = out + y
        gr = grad(dy)
        g["dx"] = g["dx"] + gr["dx"]
        g["shared"] = {n: gr[n] for n in ("dW_up", "dW_down", "db_up", "db_down")}
    return out, g


def _near(got, want, what):
    """Every value passes at most four roundings to bf16 on its way (the pre-activations, their gradient or the
    scaled activations, a partial result, the result): each 2**-9 of a value that the later sums take with its
    sign, so the whole differs by at most about 4 * 2**-9 of the terms' magnitudes; these are random, and their
    norm is within twice that of the sums' here."""
    got = got.double().cpu().numpy().reshape(want.shape)
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel < 2 * 4 * 2.0 ** -9, (what, rel)


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("act", [ob.SILU, ob.GELU])
def test_layer_against_the_oracle(gated, full, act):
    rng = np.random.default_rng(5 + gated + 2 * full)
    x, tx = bf(rng.standard_normal((T, D)))
    dy, tdy = bf(rng.standard_normal((T, D)))
    res, tres = bf(rng.standard_normal((T, D)))
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    w, sh = _weights(rng, gated, E), _weights(rng, gated, 1)
    p, seed = (0.25, 77) if full else (0.0, 1)
    gw, gs = _gpu(w), _gpu(sh)
    if not full:
        for v in (w, sh):
            v["b_up"] = (np.zeros_like(v["b_up"][0]), None)
            v["b_down"] = (np.zeros_like(v["b_down"][0]), None)
        gw["b_up"] = gw["b_down"] = None
    fw = layer.forward_bf16(tx.cuda(), gw["w_up"], gw["w_down"], logits, K, b_up=gw["b_up"], b_down=gw["b_down"], act=act,
                            shared=gs if full else None, residual=tres.cuda() if full else None, dropout=p, seed=seed)
    bw = layer.backward_bf16(fw, tdy.cuda())
    val = lambda v: {n: a[0] for n, a in v.items()}  # noqa: E731
    y, g = _reference(x, dy, val(w), val(sh) if full else None, fw["route"], act, gated, res if full else None, p, seed)
    _near(fw["y"], y, "y")
    for n in ("dx", "dW_up", "dW_down", "dg"):
        _near(bw[n], g[n], n)
    if full:
        _near(bw["db_up"], g["db_up"], "db_up")
        _near(bw["db_down"], g["db_down"], "db_down")
        for n in ("dW_up", "dW_down", "db_up", "db_down"):
            _near(bw["shared"][n], g["shared"][n], "shared " + n)
        assert torch.equal(bw["dresidual"], tdy.cuda())
    else:
        assert bw["db_up"] is None and bw["dresidual"] is None


def test_layer_gradient_against_differences():
    """<dy, y> along random directions of x and the weights, from the oracle's forward, against the backward's."""
    rng = np.random.default_rng(8)
    x, tx = bf(rng.standard_normal((T, D)))
    dy, tdy = bf(rng.standard_normal((T, D)))
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    w = _weights(rng, True, E)
    gw = _gpu(w)
    fw = layer.forward_bf16(tx.cuda(), gw["w_up"], gw["w_down"], logits, K, b_up=gw["b_up"], b_down=gw["b_down"])
    bw = layer.backward_bf16(fw, tdy.cuda())
    val = {n: a[0] for n, a in w.items()}

    def loss(dx, v):
        y, _ = _reference(x + dx, dy, v, None, fw["route"], ob.SILU, True, None, 0.0, 1)
        return (y * dy).sum()
    step = 1e-5
    for name, key in (("dx", None), ("dW_up", "w_up"), ("dW_down", "w_down"), ("db_up", "b_up"), ("db_down", "b_down")):
        grad = bw[name].double().cpu().numpy()
        u = np.sign(grad)                               # every term counts with the same sign: no cancellation
        if key is None:
            num = (loss(step * u, val) - loss(-step * u, val)) / (2 * step)
        else:
            num = (loss(0, {**val, key: val[key] + step * u}) - loss(0, {**val, key: val[key] - step * u})) / (2 * step)
        assert abs((grad * u).sum() - num) < 2 * 4 * 2.0 ** -9 * abs(num), name


def test_layer_with_router_and_balance():
    """The router's own calls behind the layer: the same as when made one by one."""
    rng = np.random.default_rng(9)
    d = 128
    x = bf(rng.standard_normal((T, d)))[1].cuda()
    dy = bf(rng.standard_normal((T, d)))[1].cuda()
    rw = bf(rng.standard_normal((E, d)) * 0.1)[1].cuda()
    wu, wd = bf(rng.standard_normal((E, 2, F, d)) * 0.1)[1].cuda(), bf(rng.standard_normal((E, d, F)) * 0.1)[1].cuda()
    db = torch.full((1,), 0.01, device="cuda")
    fw = layer.forward_bf16(x, wu, wd, None, K, router_w=rw, balance=True)
    bw = layer.backward_bf16(fw, dy, dbalance=db)
    plain = layer.backward_bf16(fw, dy)
    assert torch.equal(bw["dW_up"], plain["dW_up"]) and torch.equal(bw["dg"], plain["dg"])
    r = fw["route"]
    dl = m4.moe_balance_loss_backward(db, fw["logits"], fw["balance"]["counts"], fw["balance"]["tokens"], K, dlogits=plain["dlogits"])
    assert torch.equal(bw["dlogits"], dl)
    assert torch.equal(bw["dx"], m4.moe_unpermute_sum_router_dense(bw["dXp"], r["inv_perm"], T, K, dl, rw))
    assert torch.equal(bw["dW_router"], m4.moe_router_wgrad_dense(x, dl))
    assert torch.equal(plain["dx"], m4.moe_unpermute_sum_router(bw["dXp"], r["inv_perm"], T, K, plain["dlogits"], r["idx"], rw))


@pytest.mark.parametrize("t", [1, 64])
def test_layer_graph_replay(t):
    rng = np.random.default_rng(10)
    x, dy, res = (bf(rng.standard_normal((t, D)))[1].cuda() for _ in range(3))
    lg = torch.from_numpy(rng.standard_normal((t, E)).astype(np.float32)).cuda()
    w, sh = _gpu(_weights(rng, True, E)), _gpu(_weights(rng, True, 1))

    def step():
        fw = layer.forward_bf16(x, w["w_up"], w["w_down"], lg, K, b_up=w["b_up"], b_down=w["b_down"], shared=sh, residual=res, dropout=0.1)
        bw = layer.backward_bf16(fw, dy)
        return [fw["y"], bw["dx"], bw["dW_up"], bw["dW_down"], bw["dlogits"], bw["db_up"], bw["shared"]["dW_up"]]
    ref = [v.clone() for v in step()]
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
        for i, (a, b) in enumerate(zip(outs, ref)):
            assert torch.equal(a, b), i
        step()
        torch.cuda.synchronize()


@pytest.mark.parametrize("gated", [True, False])
def test_empty_batch(gated):
    """No tokens: empty outputs, weight gradients of zeros."""
    rng = np.random.default_rng(12)
    x = torch.empty((0, D), dtype=torch.bfloat16, device="cuda")
    w, sh = _gpu(_weights(rng, gated, E)), _gpu(_weights(rng, gated, 1))
    fw = layer.forward_bf16(x, w["w_up"], w["w_down"], torch.empty((0, E), device="cuda"), K, b_up=w["b_up"], b_down=w["b_down"],
                            shared=sh, residual=x, dropout=0.1)
    bw = layer.backward_bf16(fw, x)
    assert fw["y"].shape == (0, D) and bw["dx"].shape == (0, D) and bw["dlogits"].shape == (0, E)
    for g, v in ((bw, w), (bw["shared"], sh)):
        for n in ("w_up", "w_down", "b_up", "b_down"):
            d = g["d" + n.replace("w_", "W_")]
            assert d.shape == v[n].shape and not d.any(), n


def test_single_token_without_saving():
    """Serving: nothing kept, and the backward refuses."""
    rng = np.random.default_rng(11)
    x = bf(rng.standard_normal((1, D)))[1].cuda()
    lg = torch.from_numpy(rng.standard_normal((1, E)).astype(np.float32)).cuda()
    w = _gpu(_weights(rng, True, E))
    a = layer.forward_bf16(x, w["w_up"], w["w_down"], lg, K, save=False)
    b = layer.forward_bf16(x, w["w_up"], w["w_down"], lg, K)
    assert torch.equal(a["y"], b["y"]) and a["pre"] is None
    with pytest.raises(ValueError, match="save"):
        layer.backward_bf16(a, x)
