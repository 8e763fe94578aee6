"""Cases of the expert layer in BF16, with a plain form of each call.

The operators: the gated feed-forward block (both input projections, the
activation and the product; its backward through the output projection), the
expert-grouped BF16 product with bias, activation and residual (with its input
and weight gradients), and the combine with dropout and residual (with its
gradient).  With ``own`` false run() computes them from elementary torch
operations in 32 bits, with ``own`` true it makes the calls of
precision_moe_numerics_quant_amd.  exact() computes the same results in 64
bits from the definitions.
"""
import math

import torch

own = False

DEV = "cuda"


# -------------------------------------------------------------------- cases

def listed():
    return [
        # a training step's gated experts: x gathered through the routing, pre-activations kept for the backward
        dict(name="gated_train", op="gated", T=16384, k=8, E=384, zipf=1.1, K=4096, F=1024, act="silu", bias=False, save=True),
        # one decoded token: eight of 384 experts, one row each
        dict(name="gated_token", op="gated", T=1, k=8, E=384, zipf=0.0, K=4096, F=1024, act="silu", bias=False, save=False),
        # the training step's backward into the pre-activations: the gate-scaled gradient through the output projection
        dict(name="gated_dgrad_train", op="gated_dgrad", T=16384, k=8, E=384, zipf=1.1, N=4096, F=1024, act="silu", scale=True),
        # a short batch of few, ragged experts with odd widths
        dict(name="gated_dgrad_odd", op="gated_dgrad", T=1000, k=4, E=37, zipf=0.5, N=1032, F=344, act="gelu", scale=False),
        # a dense shared expert's output projection, with its bias, added to the routed experts' output
        dict(name="gemm_shared", op="gemm", T=16384, k=1, E=1, zipf=0.0, N=4096, K=1536, act="none", bias=True, residual=True,
             dtype="bf16", save=False, mapped=False),
        # the output projection of a rollout batch: about ten rows for each of 384 experts
        dict(name="gemm_rollout", op="gemm", T=512, k=8, E=384, zipf=0.0, N=4096, K=1024, act="none", bias=False, residual=False,
             dtype="f32", save=False, mapped=False),
        # the training step's input gradient of both input projections
        dict(name="dgrad_train", op="dgrad", T=16384, k=8, E=384, zipf=1.1, N=2048, K=4096, act="none", scale=False, dtype="f32",
             mapped=False),
        # ungated experts of a short batch: through the output projection and the activation
        dict(name="dgrad_odd", op="dgrad", T=333, k=2, E=9, zipf=0.5, N=520, K=136, act="silu", scale=True, dtype="bf16", mapped=True),
        # the training step's weight gradient of the output projections
        dict(name="wgrad_train", op="wgrad", T=16384, k=8, E=384, zipf=1.1, N=4096, K=1024, bias=False, maps="dy"),
        # a dense shared expert's weight and bias gradients
        dict(name="wgrad_shared", op="wgrad", T=16384, k=1, E=1, zipf=0.0, N=1536, K=4096, bias=True, maps="none"),
        # the layer's tail in a training step, and its gradient
        dict(name="dropout_train", op="dropout", T=16384, k=8, d=4096, p=0.1, residual=True),
        # a short sequence
        dict(name="dropout_short", op="dropout", T=37, k=2, d=1000, p=0.5, residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gated", "gated_dgrad", "gemm", "dgrad", "wgrad", "dropout"))
    if op == "dropout":
        return dict(op=op, T=_log(rng, 1, 16384), k=rng.randint(1, 8), d=4 * _log(rng, 2, 1024), p=rng.choice((0.0, 0.1, 0.5, 0.9)),
                    residual=rng.random() < 0.5)
    E = _log(rng, 1, 384)
    k = rng.randint(1, min(8, E))
    c = dict(op=op, T=_log(rng, 1, 16384), k=k, E=E, zipf=rng.choice((0.0, 0.5, 1.1)))
    wide, narrow = 8 * _log(rng, 8, 512), 8 * _log(rng, 4, 128)  # the model's and the experts' width
    act = rng.choice(("silu", "gelu"))
    if op == "gated":
        return dict(c, K=wide, F=narrow, act=act, bias=rng.random() < 0.5, save=rng.random() < 0.5)
    if op == "gated_dgrad":
        return dict(c, N=wide, F=narrow, act=act, scale=rng.random() < 0.5)
    N, K = rng.choice(((wide, narrow), (narrow, wide)))
    if op == "gemm":
        return dict(c, N=N, K=K, act=rng.choice(("none", "silu", "gelu")), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    dtype=rng.choice(("bf16", "f32")), save=rng.random() < 0.5, mapped=rng.random() < 0.5)
    if op == "dgrad":
        return dict(c, N=N, K=K, act=rng.choice(("none", "silu", "gelu")), scale=rng.random() < 0.5, dtype=rng.choice(("bf16", "f32")),
                    mapped=rng.random() < 0.5)
    return dict(c, N=N, K=K, bias=rng.random() < 0.5, maps=rng.choice(("none", "dy", "a")))


# ------------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + salt * 7919 + 17) & 0x7FFFFFFFFFFFFFFF)
    return g


def _randn(shape, g, std=1.0, dtype=torch.float32):
    """Normal values, made in parts of at most 2^27 so that a large bfloat16 tensor needs little beside it."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV) * std
    return out


BF = torch.bfloat16


def _routing(c, seed):
    """Top-k of N(0, 1) logits with a Zipf bias: gates [T, k], each row's
    assignment (perm), each assignment's row (inv) and the experts' row offsets."""
    T, E, k = c["T"], c["E"], c["k"]
    z = _randn((T, E), _gen(seed, 1))
    if c["zipf"]:
        z = z - c["zipf"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    top = torch.topk(z, k, dim=1)
    flat = top.indices.reshape(-1)
    perm = torch.argsort(flat, stable=True)
    cnt = torch.bincount(flat, minlength=E)
    off = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(cnt, 0)))
    return dict(gates=torch.softmax(top.values, 1), perm=perm.int(), off=off.int(), counts=cnt.tolist())


def prepare(case, seed):
    c = dict(case)
    op = c["op"]
    s = dict(case=c)
    if op == "dropout":
        T, k, d = c["T"], c["k"], c["d"]
        s.update(yp=_randn((T * k, d), _gen(seed, 2)), gates=torch.softmax(_randn((T, k), _gen(seed, 3)), 1),
                 inv=torch.randperm(T * k, generator=_gen(seed, 4), device=DEV).int(), dy=_randn((T, d), _gen(seed, 5), 1e-3, BF),
                 residual=_randn((T, d), _gen(seed, 6), 1.0, BF) if c["residual"] else None, seed=int(seed) + 1)
        return s
    T, k, E = c["T"], c["k"], c["E"]
    M = T * k
    r = _routing(c, seed)
    s.update(off=r["off"], counts=r["counts"], map=r["perm"])
    gates = r["gates"].reshape(-1)  # by assignment: row r of the product has the gate of assignment map[r]
    if op == "gated":
        K, F = c["K"], c["F"]
        s.update(x=_randn((T, K), _gen(seed, 2), 1.0, BF), w=_randn((E, 2, F, K), _gen(seed, 3), 0.02, BF),
                 bias=_randn((E, 2, F), _gen(seed, 4), 0.1) if c["bias"] else None)
    elif op == "gated_dgrad":
        N, F = c["N"], c["F"]
        s.update(dy=_randn((T, N), _gen(seed, 2), 1e-3, BF), w=_randn((E, N, F), _gen(seed, 3), 0.02, BF),
                 gu=_randn((M, 2, F), _gen(seed, 4), 1.0, BF), scale=gates if c["scale"] else None)
    elif op == "gemm":
        N, K = c["N"], c["K"]
        od = BF if c["dtype"] == "bf16" else torch.float32
        s.update(a=_randn((T if c["mapped"] else M, K), _gen(seed, 2), 1.0, BF), w=_randn((E, N, K), _gen(seed, 3), 0.02, BF),
                 bias=_randn((E, N), _gen(seed, 4), 0.1) if c["bias"] else None,
                 residual=_randn((M, N), _gen(seed, 5), 1.0, od) if c["residual"] else None)
        if not c["mapped"]:
            s["map"] = None
    elif op == "dgrad":
        N, K = c["N"], c["K"]
        s.update(dy=_randn((T if c["mapped"] else M, N), _gen(seed, 2), 1e-3, BF), w=_randn((E, N, K), _gen(seed, 3), 0.02, BF),
                 pre=_randn((M, K), _gen(seed, 4), 1.0, BF) if c["act"] != "none" else None, scale=gates if c["scale"] else None)
        if not c["mapped"]:
            s["map"] = None
    else:
        N, K = c["N"], c["K"]
        s.update(dy=_randn((T if c["maps"] == "dy" else M, N), _gen(seed, 2), 1e-3, BF),
                 a=_randn((T if c["maps"] == "a" else M, K), _gen(seed, 3), 1.0, BF))
    return s


# -------------------------------------------------------------- plain forms

def _act(name, x):
    """The activation and its derivative."""
    if name == "none":
        return x, torch.ones_like(x)
    if name == "silu":
        p, dp = x, 1.0
    else:  # GELU by its tanh form: x sigmoid(2 sqrt(2 / pi) (x + 0.044715 x^3))
        c = 2.0 * math.sqrt(2.0 / math.pi)
        p, dp = c * (x + 0.044715 * x * x * x), c * (1.0 + 3 * 0.044715 * x * x)
    t = 1.0 / (1.0 + torch.exp(-p))
    return x * t, t + x * t * (1.0 - t) * dp


def _experts(s):
    """Each expert with rows, and its first and last row."""
    r = 0
    for e, n in enumerate(s["counts"]):
        if n:
            yield e, r, r + n
        r += n


def _rows(s, x, a, b, mapped):
    """Rows a to b of the routed matrix, in 32 bits."""
    if not mapped:
        return x[a:b].float()
    return x[s["map"][a:b].long() // s["case"]["k"]].float()


def _scale(s, a, b, mapped):
    """Their gates, as a column (1 without)."""
    if s["scale"] is None:
        return 1.0
    return (s["scale"][s["map"][a:b].long()] if mapped else s["scale"][a:b])[:, None]


def _gated(s):
    c = s["case"]
    M, F = c["T"] * c["k"], c["F"]
    h = torch.empty((M, F), dtype=BF, device=DEV)
    gu = torch.empty((M, 2, F), dtype=BF, device=DEV) if c["save"] else None
    for e, a, b in _experts(s):
        z = _rows(s, s["x"], a, b, True) @ s["w"][e].view(2 * F, -1).float().t()
        if c["bias"]:
            z = z + s["bias"][e].view(-1)
        h[a:b] = _act(c["act"], z[:, :F])[0] * z[:, F:]
        if c["save"]:
            gu[a:b] = z.view(-1, 2, F)
    return dict(h=h, gu=gu) if c["save"] else dict(h=h)


def _gated_dgrad(s):
    c = s["case"]
    M, F = c["T"] * c["k"], c["F"]
    dgu = torch.empty((M, 2, F), dtype=BF, device=DEV)
    hs = torch.empty((M, F), dtype=BF, device=DEV)
    for e, a, b in _experts(s):
        dh = _rows(s, s["dy"], a, b, True) @ s["w"][e].float()
        g, u = s["gu"][a:b, 0].float(), s["gu"][a:b, 1].float()
        f, df = _act(c["act"], g)
        sc = _scale(s, a, b, True)
        dh, h = dh * sc, f * u * sc
        dgu[a:b, 0], dgu[a:b, 1], hs[a:b] = dh * u * df, dh * f, h
    return dict(dgu=dgu, hs=hs)


def _gemm(s):
    c = s["case"]
    out = torch.empty((c["T"] * c["k"], c["N"]), dtype=BF if c["dtype"] == "bf16" else torch.float32, device=DEV)
    pre = torch.empty(out.shape, dtype=BF, device=DEV) if c["save"] else None
    for e, a, b in _experts(s):
        z = _rows(s, s["a"], a, b, c["mapped"]) @ s["w"][e].float().t()
        if c["bias"]:
            z = z + s["bias"][e]
        if c["save"]:
            pre[a:b] = z
        z = _act(c["act"], z)[0]
        out[a:b] = z + s["residual"][a:b].float() if c["residual"] else z
    return dict(c=out, pre=pre) if c["save"] else dict(c=out)


def _dgrad(s):
    c = s["case"]
    out = torch.empty((c["T"] * c["k"], c["K"]), dtype=BF if c["dtype"] == "bf16" else torch.float32, device=DEV)
    hs = torch.empty(out.shape, dtype=BF, device=DEV) if c["act"] != "none" else None
    for e, a, b in _experts(s):
        z = _rows(s, s["dy"], a, b, c["mapped"]) @ s["w"][e].float()
        sc = _scale(s, a, b, c["mapped"])
        z = z * sc
        if hs is not None:
            f, df = _act(c["act"], s["pre"][a:b].float())
            z = z * df
            hs[a:b] = f * sc
        out[a:b] = z
    return dict(dx=out) if hs is None else dict(dx=out, hs=hs)


def _wgrad(s):
    c = s["case"]
    dw = torch.zeros((c["E"], c["N"], c["K"]), device=DEV)
    db = torch.zeros((c["E"], c["N"]), device=DEV)
    for e, a, b in _experts(s):
        dy = _rows(s, s["dy"], a, b, c["maps"] == "dy")
        dw[e] = dy.t() @ _rows(s, s["a"], a, b, c["maps"] == "a")
        if c["bias"]:
            db[e] = dy.sum(0)
    return dict(dw=dw, db=db) if c["bias"] else dict(dw=dw)


def _fmix(h):
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & 0xFFFFFFFF
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _keep(n, p, seed, stream):
    """Of each of n elements: whether it is kept (its 16 random bits under the
    key (seed, stream) are below q), and q, 65536 times the chance of that."""
    t = lambda v: torch.tensor(v, dtype=torch.int64, device=DEV)  # noqa: E731
    key = _fmix(_fmix(_fmix(t(seed & 0xFFFFFFFF)) ^ t(seed >> 32)) ^ t(stream))
    i = torch.arange(n, device=DEV)
    j = i >> 1
    w = _fmix((j & 0xFFFFFFFF) ^ _fmix(key ^ (j >> 32)))
    q = round((1.0 - p) * 65536)
    return torch.where((i & 1) == 1, w >> 16, w & 0xFFFF) < q, q


STREAM = 4


def _dropout(s):
    c = s["case"]
    T, k, d = c["T"], c["k"], c["d"]
    keep, q = _keep(T * d, c["p"], s["seed"], STREAM)
    keep = keep.view(T, d)
    y = (s["yp"][s["inv"].long()].view(T, k, d) * s["gates"][:, :, None]).sum(1)
    y = torch.where(keep, y * (65536.0 / q), torch.zeros_like(y))
    if c["residual"]:
        y = y + s["residual"].float()
    dx = s["dy"].float()
    return dict(y=y.to(BF), dx=torch.where(keep, dx * (65536.0 / q), torch.zeros_like(dx)).to(BF))


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if not own:
        return {"gated": _gated, "gated_dgrad": _gated_dgrad, "gemm": _gemm, "dgrad": _dgrad, "wgrad": _wgrad, "dropout": _dropout}[op](s)
    import precision_moe_numerics_quant_amd as m4
    if op == "dropout":
        return dict(y=m4.moe_combine_dropout(s["yp"], s["gates"], s["inv"], c["p"], s["seed"], STREAM, residual=s["residual"]),
                    dx=m4.moe_dropout_backward(s["dy"], c["p"], s["seed"], STREAM))
    dt = BF if c.get("dtype") == "bf16" else torch.float32
    act = {"none": m4.ACT_NONE, "silu": m4.ACT_SILU, "gelu": m4.ACT_GELU}[c.get("act", "none")]
    if op == "gated":
        h, gu = m4.moe_gated_gemm_bf16(s["x"], s["w"], s["off"], bias=s["bias"], act=act, row_map=s["map"], map_div=c["k"], save=c["save"])
        return dict(h=h, gu=gu) if c["save"] else dict(h=h)
    if op == "gated_dgrad":
        dgu, hs = m4.moe_gated_gemm_bf16_dgrad(s["dy"], s["w"], s["gu"], s["off"], act=act, row_scale=s["scale"], row_map=s["map"],
                                               map_div=c["k"])
        return dict(dgu=dgu, hs=hs)
    if op == "gemm":
        out, pre = m4.moe_grouped_gemm_bf16(s["a"], s["w"], s["off"], bias=s["bias"], act=act, residual=s["residual"], row_map=s["map"],
                                            map_div=c["k"] if c["mapped"] else 1, out_dtype=dt, save_pre=c["save"])
        return dict(c=out, pre=pre) if c["save"] else dict(c=out)
    if op == "dgrad":
        dx, hs = m4.moe_grouped_gemm_bf16_dgrad(s["dy"], s["w"], s["off"], pre=s["pre"], act=act, row_scale=s["scale"], row_map=s["map"],
                                                map_div=c["k"] if c["mapped"] else 1, out_dtype=dt)
        return dict(dx=dx) if hs is None else dict(dx=dx, hs=hs)
    dw, db = m4.moe_grouped_gemm_bf16_wgrad(s["dy"], s["a"], s["off"], dy_map=s["map"] if c["maps"] == "dy" else None,
                                            a_map=s["map"] if c["maps"] == "a" else None, map_div=c["k"] if c["maps"] != "none" else 1,
                                            bias_grad=c["bias"])
    return dict(dw=dw, db=db) if c["bias"] else dict(dw=dw)


# --------------------------------------------------------------------- work

def work(case):
    c = case
    op = c["op"]
    if op == "dropout":
        T, k, d = c["T"], c["k"], c["d"]
        return {"bytes": T * k * (4 * d + 8) + T * d * (2 * 3 + (2 if c["residual"] else 0)), "flops": T * d * (2 * k + 4)}
    M = c["T"] * c["k"]
    # the weights of every expert that may have a row (fewer have one where the routing is skewed)
    experts = min(c["E"], M)
    if op == "gated":
        K, F = c["K"], c["F"]
        n = c["T"] * K * 2 + M * 4 + experts * 2 * F * (2 * K + (4 if c["bias"] else 0)) + M * F * (6 if c["save"] else 2)
        return {"bytes": n, "flops": 4 * M * F * K}
    if op == "gated_dgrad":
        N, F = c["N"], c["F"]
        n = c["T"] * N * 2 + M * 4 + experts * N * F * 2 + M * F * 10 + (M * 4 if c["scale"] else 0)
        return {"bytes": n, "flops": 2 * M * F * N}
    N, K = c["N"], c["K"]
    o = 2 if c.get("dtype") == "bf16" else 4
    if op == "gemm":
        n = (c["T"] * K * 2 + M * 4 if c["mapped"] else M * K * 2) + experts * N * (2 * K + (4 if c["bias"] else 0))
        return {"bytes": n + M * N * (o + (o if c["residual"] else 0) + (2 if c["save"] else 0)), "flops": 2 * M * N * K}
    if op == "dgrad":
        n = (c["T"] * N * 2 + M * 4 if c["mapped"] else M * N * 2) + experts * N * K * 2 + (M * 4 if c["scale"] else 0)
        return {"bytes": n + M * K * (o + (4 if c["act"] != "none" else 0)), "flops": 2 * M * N * K}
    n = (c["T"] if c["maps"] == "dy" else M) * N * 2 + (c["T"] if c["maps"] == "a" else M) * K * 2 + c["E"] * N * K * 4
    return {"bytes": n + (M * 4 if c["maps"] != "none" else 0) + (c["E"] * N * 4 if c["bias"] else 0), "flops": 2 * M * N * K}


# -------------------------------------------------------------------- exact

def _d_sigmoid(name, x):
    """The factor of x in the activation, and the activation's derivative, in 64 bits."""
    if name == "none":
        return torch.ones_like(x), torch.ones_like(x)
    if name == "silu":
        t = torch.sigmoid(x)
        return t, t * (1 + x * torch.sigmoid(-x))
    inner = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    th = torch.tanh(inner)
    return 0.5 * (1 + th), 0.5 * (1 + th) + 0.5 * x * (1 - th * th) * math.sqrt(2 / math.pi) * (1 + 0.134145 * x * x)


def _exact_rows(s, x, a, b, mapped):
    if not mapped:
        return x[a:b].double()
    return x.index_select(0, torch.div(s["map"][a:b], s["case"]["k"], rounding_mode="floor")).double()


def _exact_product(s):
    c = s["case"]
    op = c["op"]
    M = c["T"] * c["k"]
    off = s["off"].tolist()
    spans = [(e, a, b) for e, (a, b) in enumerate(zip(off[:-1], off[1:])) if b > a]
    new = lambda *n: torch.empty(n, dtype=torch.float64, device=DEV)  # noqa: E731
    if op == "gated":
        F = c["F"]
        h, gu = new(M, F), new(M, 2, F) if c["save"] else None
        for e, a, b in spans:
            x = _exact_rows(s, s["x"], a, b, True)
            z = [torch.mm(x, s["w"][e, i].double().t()) + (s["bias"][e, i].double() if c["bias"] else 0) for i in (0, 1)]
            h[a:b] = z[0] * _d_sigmoid(c["act"], z[0])[0] * z[1]
            if c["save"]:
                gu[a:b] = torch.stack(z, 1)
        return dict(h=h, gu=gu) if c["save"] else dict(h=h)
    if op == "gated_dgrad":
        F = c["F"]
        dgu, hs = new(M, 2, F), new(M, F)
        for e, a, b in spans:
            w = s["scale"].double().index_select(0, s["map"][a:b])[:, None] if c["scale"] else 1.0
            dh = w * torch.mm(_exact_rows(s, s["dy"], a, b, True), s["w"][e].double())
            g, u = s["gu"][a:b].double().unbind(1)
            f, df = _d_sigmoid(c["act"], g)
            dgu[a:b] = torch.stack((dh * u * df, dh * g * f), 1)
            hs[a:b] = w * g * f * u
        return dict(dgu=dgu, hs=hs)
    N, K = c["N"], c["K"]
    if op == "gemm":
        out, pre = new(M, N), new(M, N) if c["save"] else None
        for e, a, b in spans:
            z = torch.mm(_exact_rows(s, s["a"], a, b, c["mapped"]), s["w"][e].double().t())
            z = z + (s["bias"][e].double() if c["bias"] else 0)
            if c["save"]:
                pre[a:b] = z
            out[a:b] = z * _d_sigmoid(c["act"], z)[0] + (s["residual"][a:b].double() if c["residual"] else 0)
        return dict(c=out, pre=pre) if c["save"] else dict(c=out)
    if op == "dgrad":
        out, hs = new(M, K), new(M, K) if c["act"] != "none" else None
        for e, a, b in spans:
            rows = s["map"][a:b].long() if c["mapped"] else slice(a, b)
            w = s["scale"].double()[rows][:, None] if c["scale"] else 1.0
            z = w * torch.mm(_exact_rows(s, s["dy"], a, b, c["mapped"]), s["w"][e].double())
            if hs is not None:
                x = s["pre"][a:b].double()
                f, df = _d_sigmoid(c["act"], x)
                z, hs[a:b] = z * df, w * x * f
            out[a:b] = z
        return dict(dx=out) if hs is None else dict(dx=out, hs=hs)
    dw = torch.zeros((c["E"], N, K), dtype=torch.float64, device=DEV)
    db = torch.zeros((c["E"], N), dtype=torch.float64, device=DEV)
    for e, a, b in spans:
        dy = _exact_rows(s, s["dy"], a, b, c["maps"] == "dy")
        dw[e] = torch.mm(dy.t().contiguous(), _exact_rows(s, s["a"], a, b, c["maps"] == "a"))
        db[e] = torch.ones(b - a, dtype=torch.float64, device=DEV) @ dy
    return dict(dw=dw, db=db) if c["bias"] else dict(dw=dw)


def _exact_dropout(s):
    c = s["case"]
    T, k, d = c["T"], c["k"], c["d"]
    M32 = (1 << 32) - 1

    def mix(h):
        for mul, sh in ((0x85EBCA6B, 16), (0xC2B2AE35, 13)):
            h = ((h ^ (h >> sh)) * mul) & M32
        return h ^ (h >> 16)
    base = mix(mix(mix(s["seed"] & M32) ^ (s["seed"] >> 32)) ^ STREAM)
    q = round((1.0 - c["p"]) * 65536)
    word = mix(torch.arange((T * d + 1) // 2, device=DEV) ^ mix(base))  # (fewer than 2^32 pairs)
    keep = (torch.stack((word & 0xFFFF, word >> 16), 1).view(-1)[:T * d] < q).view(T, d)
    y = torch.zeros((T, d), dtype=torch.float64, device=DEV)
    for j in range(k):
        y += s["gates"][:, j, None].double() * s["yp"].index_select(0, s["inv"].view(T, k)[:, j]).double()
    y = y * keep * (65536 / q)
    if c["residual"]:
        y = y + s["residual"].double()
    return dict(y=y, dx=s["dy"].double() * keep * (65536 / q))


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_dropout(s) if case["op"] == "dropout" else _exact_product(s)
