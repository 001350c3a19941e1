"""Workloads of the router with its balance loss, the clipping of the gradients and the layer on 4-bit weights.

``run`` computes a workload's operator either with plain torch operations in 32 bits
(``own = False``) or with the library's entry points (``own = True``).  Sizes follow the
routing workloads of ``ep_inputs.py`` (hidden 7168 or 4096, top-8 of 64 to 256 experts, 128 to
16384 tokens); the experts' inner width is 2048, or an uneven 1400 or 1408.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu", "swiglu", "geglu")  # in the order of the EP_ACT_* codes
SCORES = ("softmax", "sigmoid")                             # in the order of the EP_SCORE_* codes
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)             # values of the 4-bit codes 0..7; codes 8..15 are their negatives

ROUTE = dict(T=1, E=8, K=1, score="softmax", normalise=True, scale=1.0, bf16=False, bias=False, stats=False, dweights=True,
             masked=0.0)
CLIP = dict(layers=1, E=1, H=64, I=64, odd=False, clipped=True)
FP4 = dict(T=1, H=256, I=256, E=1, K=1, R=1, act="none", bias=False, residual=False, empty=0.0)


def _case(kind, name=None, **kw):
    base = ROUTE if kind in ("route", "balance", "route_backward") else CLIP if kind == "clip" else FP4
    c = {"kind": kind, **base, **kw}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # the router of a decode batch, before the few-token layer
        _case("route", "route-128", T=128, E=256, K=8, bf16=True),
        # the router of a training step: sigmoid scores, a selection bias, and the balance statistics with it
        _case("route", "route-16384-bias", T=16384, E=256, K=8, score="sigmoid", scale=2.5, bias=True, stats=True),
        # the balance loss of choices that were made elsewhere, on a short padded batch over an odd number of experts
        _case("balance", "balance-1000", T=1000, E=127, K=4, bf16=True, masked=0.1),
        # the same for a training step
        _case("balance", "balance-16384", T=16384, E=64, K=8),
        # the router's gradient on a short padded batch
        _case("route_backward", "route-backward-1000", T=1000, E=127, K=4, score="sigmoid", bf16=True, masked=0.1),
        # the router's gradient in a training step: from the combine's weights and both losses
        _case("route_backward", "route-backward-16384", T=16384, E=256, K=8),
        # the gradients of a small model of eight layers: many small tensors, back to back in one buffer
        _case("clip", "clip-40-tensors", layers=8, E=8, H=136, I=72, odd=True),
        # one layer's experts in a training step
        _case("clip", "clip-experts", layers=1, E=32, H=7168, I=2048),
        # a shared expert's up projection for one token: a matrix-vector product
        _case("product_fp4", "fp4-1-swiglu", T=1, H=7168, I=2048, act="swiglu"),
        # a decode batch's up projection over all experts, on the rows that the dispatch left
        _case("product_fp4", "fp4-100-swiglu", T=100, H=4096, I=1408, E=128, K=8, R=4, act="swiglu", bias=True),
        # one token being generated
        _case("tokens_fp4", "tokens-fp4-1", T=1, H=7168, I=2048, E=64, K=8, act="swiglu", residual=True),
        # the decode batch: nearly every expert is reached by a few tokens
        _case("tokens_fp4", "tokens-fp4-128", T=128, H=7168, I=2048, E=256, K=8, act="swiglu"),
    ]


def _spread(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high + 1)))
    return max(low, min(high, int(v))) // step * step


def draw(rng):
    kind = rng.choice(("route", "balance", "route_backward", "clip", "product_fp4", "tokens_fp4", "tokens_fp4"))
    while True:
        if kind == "clip":
            c = _case(kind, layers=_spread(rng, 1, 12), E=_spread(rng, 1, 64), H=_spread(rng, 8, 7168, 8),
                      I=_spread(rng, 8, 2048, 8), odd=rng.random() < 0.5, clipped=rng.random() < 0.75)
            if work(c)["bytes"] <= 5.6e9:
                return c
        elif kind.endswith("fp4"):
            dense = kind == "product_fp4" and rng.random() < 0.4
            E = 1 if dense else 2 ** rng.randint(2, 8)
            c = _case(kind, T=_spread(rng, 1, 128), H=_spread(rng, 128, 7168, 32), I=_spread(rng, 128, 4096, 32), E=E,
                      K=1 if dense else rng.randint(1, min(8, E)), R=1 if dense else 2 ** rng.randint(0, 2),
                      act=rng.choice(ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                      empty=0.0 if dense else rng.choice((0.0, 0.0, 0.1)))
            if E * _width(c) * c["H"] <= 7.5e9 and work(c)["bytes"] <= 5.5e9:
                return c
        else:
            E = rng.choice((_spread(rng, 4, 256), 2 ** rng.randint(2, 8), _spread(rng, 256, 1024)))
            c = _case(kind, T=_spread(rng, 1, 65536), E=E, K=rng.randint(1, min(8, E)), score=rng.choice(SCORES),
                      normalise=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)), bf16=rng.random() < 0.5,
                      bias=kind == "route" and rng.random() < 0.5, stats=kind == "route" and rng.random() < 0.6,
                      dweights=rng.random() < 0.8, masked=rng.choice((0.0, 0.0, 0.1)))
            if c["T"] * E <= 16384 * 256:
                return c


def _width(c):
    """Rows of an expert's first weight: both halves of a gated activation."""
    return c["I"] * (2 if c["act"] in ("swiglu", "geglu") else 1)


def _shapes(c):
    """The gradients of a layer: the router's and the experts' weights in bf16, their biases in fp32."""
    E, H, I = c["E"], c["H"], c["I"]
    one = [((E, H), torch.bfloat16), ((E, 2 * I, H), torch.bfloat16), ((E, 2 * I), torch.float32),
           ((E, H, I), torch.bfloat16), ((E, H), torch.float32)]
    return one * c["layers"]


def work(c):
    if c["kind"] == "clip":
        n = [math.prod(s) * (2 if t == torch.bfloat16 else 4) for s, t in _shapes(c)]
        return {"bytes": 2 * sum(n), "flops": sum(3 * math.prod(s) for s, _ in _shapes(c))}
    T, E, K = c["T"], c["E"], c["K"]
    if "H" not in c:
        logits = T * E * (2 if c["bf16"] else 4)
        if c["kind"] == "route":
            return {"bytes": logits + T * K * 8 + (E * 8 if c["stats"] else 0), "flops": T * E * 6}
        if c["kind"] == "balance":
            return {"bytes": logits + T * K * 4 + E * 8, "flops": T * E * 6}
        return {"bytes": 2 * logits + T * K * (8 if c["dweights"] else 4) + E * 4, "flops": T * E * 12}
    H, I, M = c["H"], c["I"], _width(c)
    rows = T * K * (1 - c["empty"])
    touched = E * (1 - (1 - min(1.0, K / E)) ** T)  # experts that a uniform router reaches
    el = 0.5 + 1 / 32
    if c["kind"] == "product_fp4":
        by = rows * H * 2 + rows * I * 2 * (2 if c["residual"] else 1) + touched * M * H * el
        return {"bytes": int(by), "flops": int(2 * rows * M * H)}
    by = touched * (M * H + H * I) * el + T * H * 2 * (3 if c["residual"] else 2)
    return {"bytes": int(by), "flops": int(2 * rows * (M * H + H * I))}


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    t = torch.randn(*shape, device="cuda", generator=g, dtype=dtype)
    return t.mul_(scale) if scale != 1.0 else t


def _mask(c, g):
    """1 for a token, 0 for padding, whose logits hold whatever was there: here NaN in half of them."""
    if not c["masked"]:
        return None
    return (torch.rand(c["T"], device="cuda", generator=g) >= c["masked"]).to(torch.uint8)


def _prepare_router(c, g):
    T, E, K = c["T"], c["E"], c["K"]
    dev = dict(device="cuda")
    logits = _normal(g, T, E, scale=1.5, dtype=torch.float32)
    logits += _normal(g, E, scale=0.5, dtype=torch.float32)  # some experts are more popular
    mask = _mask(c, g)
    s = {"case": c, "mask": mask}
    if mask is not None:
        noise = torch.rand(T, device="cuda", generator=g) < 0.5
        logits[(mask == 0) & noise] = float("nan")
    s["logits"] = logits.to(torch.bfloat16) if c["bf16"] else logits
    s["bias"] = _normal(g, E, scale=0.1, dtype=torch.float32) if c["bias"] else None
    if c["kind"] == "route":
        s["idx"] = torch.empty(T, K, dtype=torch.int32, **dev)
        s["w"] = torch.empty(T, K, **dev)
    else:  # the choices of a router with a little noise of its own
        noisy = logits.nan_to_num(0.0) + _normal(g, T, E, scale=0.1, dtype=torch.float32)
        idx = noisy.topk(K, 1).indices.int()
        if mask is not None:
            idx[mask == 0] = -1
        s["idx"] = idx.contiguous()
    if c["kind"] == "route_backward":
        live = torch.ones(T, device="cuda", dtype=torch.uint8) if mask is None else mask
        s["tokens"] = live.sum(dtype=torch.int32).view(1)
        flat = s["idx"].flatten().long()
        s["count"] = torch.bincount(flat[flat >= 0], minlength=E).int()
        s["dw"] = _normal(g, T, K, dtype=torch.float32) if c["dweights"] else None
        s["dlosses"] = torch.tensor([0.01, 0.001], device="cuda")  # coefficients of the losses
        s["dlogits"] = torch.empty_like(s["logits"])
    else:
        s["count"], s["tokens"] = torch.empty(E, dtype=torch.int32, **dev), torch.empty(1, dtype=torch.int32, **dev)
        s["prob"], s["losses"] = torch.empty(E, **dev), torch.empty(2, **dev)
    return s


def _prepare_clip(c, g):
    """The gradients, each of another size of values, and where they go; `odd` packs them with no regard to alignment."""
    grads, outs = [], []
    shapes = _shapes(c)
    pools = {}
    if c["odd"]:
        for t in (torch.bfloat16, torch.float32):
            n = sum(math.prod(s) + 1 for s, k in shapes if k == t)
            pools[t] = [torch.zeros(n, device="cuda", dtype=t), torch.zeros(n, device="cuda", dtype=t), 0]
    total = 0.0
    for i, (shape, t) in enumerate(shapes):
        n = math.prod(shape)
        size = 2.0 ** (i % 7 - 10)
        total += n * size * size
        if c["odd"]:
            pool = pools[t]
            pool[2] += 1
            a, b = (x[pool[2]:pool[2] + n].view(shape) for x in pool[:2])
            pool[2] += n
            a.copy_(_normal(g, *shape, scale=size, dtype=t))
        else:
            a, b = _normal(g, *shape, scale=size, dtype=t), torch.empty(shape, device="cuda", dtype=t)
        grads.append(a)
        outs.append(b)
    return {"case": c, "grads": grads, "outs": outs, "max_norm": math.sqrt(total) * (0.3 if c["clipped"] else 3.0),
            "square_sum": torch.empty(1, device="cuda", dtype=torch.float64), "norm": torch.empty(1, device="cuda")}


def _mxfp4(v):
    """Codes (two a byte, the even column's in the low half) and scale bytes (2^(byte - 127), one for 32 columns)."""
    R, C = v.shape
    v = v.float().view(R, C // 32, 32)
    top = torch.frexp(v.abs().amax(-1, keepdim=True).clamp_min(1e-30)).exponent - 1 - 2
    u = torch.ldexp(v, -top)
    code = torch.bucketize(u.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)).to(torch.uint8)
    code = (code + 8 * (u < 0)).to(torch.uint8).view(R, C // 2, 2)
    return code[..., 0] | code[..., 1] << 4, (top[..., 0] + 127).to(torch.uint8)


def _weight(g, E, M, C):
    codes = torch.empty(E, M, C // 2, device="cuda", dtype=torch.uint8)
    sf = torch.empty(E, M, C // 32, device="cuda", dtype=torch.uint8)
    for e in range(E):
        codes[e], sf[e] = _mxfp4(_normal(g, M, C, scale=C ** -0.5))
    return codes, sf


def _prepare_fp4(c, g):
    T, H, I, E, K, R = c["T"], c["H"], c["I"], c["E"], c["K"], c["R"]
    M = _width(c)
    top = torch.randn(T, E, device="cuda", generator=g).topk(K, 1)
    idx, w = top.indices.int().contiguous(), torch.softmax(top.values.float(), 1).contiguous()
    if c["empty"]:  # padded tokens name no expert
        idx[torch.rand(T, device="cuda", generator=g) < c["empty"]] = -1
    s = {"case": c, "idx": idx, "w": w}
    if c["kind"] == "tokens_fp4":
        s["x"] = _normal(g, T, H)
        s["w1"], s["s1"] = _weight(g, E, M, H)
        s["w2"], s["s2"] = _weight(g, E, H, I)
        s["b1"] = _normal(g, E, M, dtype=torch.float32) if c["bias"] else None
        s["b2"] = _normal(g, E, H, dtype=torch.float32) if c["bias"] else None
        s["residual"] = _normal(g, T, H) if c["residual"] else None
        s["out"] = torch.empty(T, H, device="cuda", dtype=torch.bfloat16)
        return s
    # the rows that the layout gives each expert: consecutive in its rank's slice
    S, L = T * K, E // R
    flat = idx.flatten().long()
    count = torch.bincount(flat[flat >= 0], minlength=E)
    first = count.cumsum(0) - count
    offset = first - first[::L].repeat_interleave(L)
    s["count"], s["offset"] = count.int(), offset.int().contiguous()
    s["S"] = S
    base = [e // L * S + o for e, o in enumerate(offset.tolist())]
    s["spans"] = [(e, b, b + n) for e, (b, n) in enumerate(zip(base, count.tolist())) if n]
    s["x"] = _normal(g, R * S, H)
    s["w1"], s["s1"] = _weight(g, E, M, H)
    s["b1"] = _normal(g, E, M, dtype=torch.float32) if c["bias"] else None
    s["residual"] = _normal(g, R * S, I) if c["residual"] else None
    s["out"] = torch.zeros(R * S, I, device="cuda", dtype=torch.bfloat16)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["kind"] == "clip":
        return _prepare_clip(case, g)
    return _prepare_fp4(case, g) if case["kind"].endswith("fp4") else _prepare_router(case, g)


def _live(s):
    """[T, 1], whether a token counts, and the logits in 32 bits with zeros in the others."""
    logits = s["logits"].float()
    live = torch.ones_like(logits[:, :1], dtype=torch.bool) if s["mask"] is None else (s["mask"] != 0).view(-1, 1)
    return live, torch.where(live, logits, torch.zeros_like(logits))


def _softmax(v):
    e = torch.exp(v - v.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _probabilities(c, logits):
    """The scores, and the probabilities of the balance loss."""
    if c["score"] == "softmax":
        p = _softmax(logits)
        return p, p
    s = 1 / (1 + torch.exp(-logits))
    return s, s / s.sum(-1, keepdim=True)


def _plain_stats(s, live, logits):
    """The counts, the sums of the probabilities, and the losses; the long sums in 64 bits."""
    c = s["case"]
    E, K = c["E"], c["K"]
    idx = torch.where(live, s["idx"].long(), -1)
    s["count"].copy_((idx.flatten()[:, None] == torch.arange(E, device="cuda")).sum(0) if idx.numel() * E < 1 << 26 else
                     torch.bincount(idx[idx >= 0], minlength=E))
    s["tokens"].copy_(live.sum().view(1))
    p = _probabilities(c, logits)[1]
    s["prob"].copy_((p.double() * live).sum(0))
    top = logits.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(logits - top).sum(-1, keepdim=True))
    V = live.sum().double().clamp_min(1)
    s["losses"][0] = (s["count"].double() * (p.double() * live).sum(0)).sum() * E / (K * V * V)
    s["losses"][1] = ((lse.double() ** 2) * live).sum() / V
    return [s["count"], s["tokens"], s["prob"], s["losses"]]


def _plain_route(s):
    c = s["case"]
    live, logits = _live(s)
    score = _probabilities(c, logits)[0]
    if s["bias"] is None:
        key = logits  # scores rise with the logits
    else:  # in 64 bits: two experts' sums may be neighbours
        key = _probabilities(c, logits.double())[0] + s["bias"].double()
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["K"]]
    w = score.gather(1, idx)
    if c["normalise"]:
        w = _softmax(logits.gather(1, idx)) if c["score"] == "softmax" else w / w.sum(-1, keepdim=True)
    s["idx"].copy_(torch.where(live, idx, -1))
    s["w"].copy_(w * c["scale"] * live)
    return [s["idx"], s["w"]] + (_plain_stats(s, live, logits) if c["stats"] else [])


def _plain_route_backward(s):
    c = s["case"]
    E, K = c["E"], c["K"]
    live, logits = _live(s)
    score, p = _probabilities(c, logits)
    V = s["tokens"].float()
    db, dz = s["dlosses"][0], s["dlosses"][1]
    b = db * E / (K * V * V) * s["count"].float()
    d = p * (b - (p * b).sum(-1, keepdim=True))
    if c["score"] == "sigmoid":
        d = d * (1 - score)
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(-1, keepdim=True)
    d = d + dz * 2 / V * (top + torch.log(total)) * (e / total)
    if s["dw"] is not None:
        at = s["idx"].long().clamp_min(0)
        sel = score.gather(1, at)
        dw = s["dw"] * c["scale"]
        if c["normalise"]:
            u = sel / sel.sum(-1, keepdim=True)
            ds = u * (dw - (u * dw).sum(-1, keepdim=True))
            if c["score"] == "sigmoid":
                ds = ds * (1 - sel)
        elif c["score"] == "sigmoid":
            ds = dw * sel * (1 - sel)
        else:
            d = d - score * (dw * sel).sum(-1, keepdim=True)
            ds = dw * sel
        d = d.scatter_add(1, at, ds)
    s["dlogits"].copy_(torch.where(live, d, torch.zeros_like(d)))
    return s["dlogits"]


def _plain_clip(s):
    total = sum(g.float().square().sum(dtype=torch.float64) for g in s["grads"])
    norm = total.sqrt().float()
    s["norm"].copy_(norm.view(1))
    factor = (s["max_norm"] / norm).clamp_max(1.0)
    for g, o in zip(s["grads"], s["outs"]):
        o.copy_(g.float() * factor)
    return [s["norm"], s["outs"]]


def _wide(codes, sf):
    """The values of 4-bit codes with one scale for each 32 columns."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(sf.float() - 127).repeat_interleave(32, -1)


def _act(name, v):
    """The activation of pre-activations `v`, its last dimension halved where it is gated."""
    if name == "none":
        return v
    if name == "relu":
        return v.clamp_min(0)
    if name in ("swiglu", "geglu"):
        a, b = v.chunk(2, -1)
        return _act("silu" if name == "swiglu" else "gelu", a) * b
    return v * torch.sigmoid(v) if name == "silu" else v * 0.5 * (1 + torch.erf(v * 0.5 ** 0.5))


def _plain_product(s):
    c = s["case"]
    for e, lo, hi in s["spans"]:
        v = s["x"][lo:hi].float() @ _wide(s["w1"][e], s["s1"][e]).t()
        if s["b1"] is not None:
            v = v + s["b1"][e]
        v = _act(c["act"], v)
        if s["residual"] is not None:
            v = v + s["residual"][lo:hi].float()
        s["out"][lo:hi] = v.bfloat16()
    return s["out"]


def _plain_tokens(s):
    c = s["case"]
    acc = torch.zeros_like(s["x"], dtype=torch.float32) if s["residual"] is None else s["residual"].float()
    for e in s["idx"].unique().tolist():
        if e < 0:
            continue
        t, j = (s["idx"] == e).nonzero(as_tuple=True)
        v = s["x"][t].float() @ _wide(s["w1"][e], s["s1"][e]).t()
        if s["b1"] is not None:
            v = v + s["b1"][e]
        v = _act(c["act"], v) @ _wide(s["w2"][e], s["s2"][e]).t()
        if s["b2"] is not None:
            v = v + s["b2"][e]
        acc[t] += v * s["w"][t, j, None]  # a router names an expert once for a token
    return acc.bfloat16()


def _own(s):
    import combine_ep_get_amd as ep

    c = s["case"]
    kind = c["kind"]
    if kind == "clip":
        if "list" not in s:  # addresses and sizes, and the workspace: laid out once, as a training loop keeps them
            s["list"] = ep.Grads.make(s["grads"], s["outs"])
            s["workspace"] = torch.empty(ep.ep_grad_workspace_bytes(s["list"]), device="cuda", dtype=torch.uint8)
        ep.ep_grad_square_sum(s["list"], s["square_sum"], s["workspace"])
        ep.ep_grad_clip(s["list"], s["square_sum"], s["max_norm"], s["norm"])
        return [s["norm"], s["outs"]]
    if kind.endswith("fp4"):
        p = ep.Problem.make(c["T"], c["H"], c["E"], c["K"], c["R"], 1, 1, s.get("S", c["T"] * c["K"]))
        q = ep.Product.make(c["H"], c["I"], ACTS.index(c["act"]))
        if kind == "product_fp4":
            seg = (None, None) if c["E"] == 1 and c["K"] == 1 else (s["count"], s["offset"])
            ep.ep_expert_product_fp4(p, q, s["x"], *seg, s["w1"], s["s1"], s["b1"], s["residual"], s["out"])
            return s["out"]
        if "workspace" not in s:
            s["workspace"] = torch.empty(ep.ep_moe_tokens_workspace_bytes(p, q), device="cuda", dtype=torch.uint8)
        ep.ep_moe_tokens_fp4(p, q, s["x"], s["idx"], s["w"], s["w1"], s["s1"], s["b1"], s["w2"], s["s2"], s["b2"],
                             s["residual"], s["out"], s["workspace"])
        return s["out"]
    # the receive buffer's fields of the problem are not used by the router
    p = ep.Problem.make(c["T"], 4096, c["E"], c["K"], 1 if c["E"] <= 256 else c["E"], 1, 1, 1)
    r = ep.Router.make(SCORES.index(c["score"]), c["normalise"], c["scale"], c["bf16"])
    if kind == "route_backward":
        ep.ep_route_backward(p, r, s["logits"], s["idx"], s["mask"], s["count"], s["tokens"], s["dw"], s["dlosses"],
                             s["dlogits"])
        return s["dlogits"]
    if "workspace" not in s:
        s["workspace"] = torch.empty(ep.ep_route_workspace_bytes(p, r), device="cuda", dtype=torch.uint8)
    stats = [s["count"], s["tokens"], s["prob"], s["losses"]]
    if kind == "balance":
        ep.ep_balance_loss(p, r, s["logits"], s["idx"], s["mask"], *stats, s["workspace"])
        return stats
    if not c["stats"]:
        ep.ep_route(p, r, s["logits"], s["bias"], s["mask"], s["idx"], s["w"])
        return [s["idx"], s["w"]]
    ep.ep_route(p, r, s["logits"], s["bias"], s["mask"], s["idx"], s["w"], *stats, s["workspace"])
    return [s["idx"], s["w"]] + stats


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "balance":
        return _plain_stats(state, *_live(state))
    return {"route": _plain_route, "route_backward": _plain_route_backward, "clip": _plain_clip,
            "product_fp4": _plain_product, "tokens_fp4": _plain_tokens}[kind](state)


def _scores64(c, v):
    """Scores and probabilities of logits in 64 bits."""
    if c["score"] == "sigmoid":
        sc = torch.special.expit(v)
        return sc, sc / torch.linalg.vector_norm(sc, 1, dim=1, keepdim=True)
    sc = torch.exp(v - torch.logsumexp(v, 1, keepdim=True))
    return sc, sc


def _losses64(c, v, rows, idx, count):
    """Balance and z loss of the rows `v` of tokens that count."""
    p = _scores64(c, v)[1]
    V = max(1, v.shape[0])
    share = p.sum(0) / V
    balance = c["E"] * torch.dot(count.to(torch.float64) / (c["K"] * V), share)
    return p.sum(0), torch.stack([balance, torch.logsumexp(v, 1).square().sum() / V])


def _exact_router(c, s):
    T, E, K = c["T"], c["E"], c["K"]
    rows = torch.arange(T, device="cuda") if s["mask"] is None else s["mask"].nonzero()[:, 0]
    v = s["logits"][rows].to(torch.float64)
    out = []
    idx = s["idx"]
    if c["kind"] == "route":
        sc = _scores64(c, v)[0]
        key = v.clone() if s["bias"] is None else sc + s["bias"].to(torch.float64)
        idx = torch.full((T, K), -1, device="cuda", dtype=torch.int32)
        w = torch.zeros(T, K, device="cuda", dtype=torch.float64)
        lane = torch.arange(E, device="cuda")
        for j in range(K):  # the greatest key that is left, of equal ones the first
            best = torch.where(key == key.amax(1, keepdim=True), lane, E).amin(1)
            idx[rows, j] = best.int()
            w[rows, j] = sc.gather(1, best[:, None])[:, 0]
            key.scatter_(1, best[:, None], -math.inf)
        if c["normalise"]:
            w[rows] = w[rows] / w[rows].sum(1, keepdim=True)
        out = [idx, w * c["scale"]]
        if not c["stats"]:
            return out
    if c["kind"] != "route_backward":
        count = torch.zeros(E + 1, device="cuda", dtype=torch.int32)
        hit = idx[rows].flatten().long()
        count.index_add_(0, torch.where(hit < 0, E, hit), torch.ones_like(hit, dtype=torch.int32))
        prob, losses = _losses64(c, v, rows, idx, count[:E])
        return out + [count[:E].contiguous(), torch.tensor([rows.numel()], device="cuda", dtype=torch.int32), prob, losses]
    # the gradient by differentiation, not by its formula
    with torch.enable_grad():
        v = v.requires_grad_()
        sc = _scores64(c, v)[0]
        total = (_losses64(c, v, rows, idx, s["count"])[1] * s["dlosses"].to(torch.float64)).sum()
        if s["dw"] is not None:
            w = sc.gather(1, idx[rows].long())
            w = w / w.sum(1, keepdim=True) if c["normalise"] else w
            total = total + (w * c["scale"] * s["dw"][rows].to(torch.float64)).sum()
        d, = torch.autograd.grad(total, v)
    full = torch.zeros(T, E, device="cuda", dtype=torch.float64)
    full[rows] = d
    return full


def _double(codes, sf):
    """float64 values of codes: sign, two bits of exponent, one of mantissa."""
    R, B = codes.shape
    nibble = torch.empty(R, B, 2, device="cuda", dtype=torch.int64)
    nibble[..., 0] = codes % 16
    nibble[..., 1] = codes // 16
    sign, ex, m = 1 - 2 * (nibble // 8), nibble // 2 % 4, nibble % 2
    v = torch.where(ex > 0, (2 + m) * 2 ** ex.clamp_min(1), 2 * m).to(torch.float64) / 4 * sign
    return (v.view(R, B // 16, 32) * torch.ldexp(torch.ones_like(sf, dtype=torch.float64), sf.int() - 127)[..., None]).view(R, 2 * B)


def _activation64(name, v):
    half = v.shape[1] // 2
    if name in ("silu", "swiglu"):
        gate = v if name == "silu" else v[:, :half]
        a = gate / (1 + torch.exp(-gate))
    elif name in ("gelu", "geglu"):
        gate = v if name == "gelu" else v[:, :half]
        a = gate * torch.special.ndtr(gate)
    else:
        a = torch.where(v > 0, v, torch.zeros_like(v)) if name == "relu" else v
    return a * v[:, half:] if name in ("swiglu", "geglu") else a


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["kind"] == "clip":
        total = torch.zeros((), device="cuda", dtype=f64)
        for g in s["grads"]:
            for part in g.flatten().split(1 << 27):
                total += torch.linalg.vector_norm(part.to(f64)) ** 2
        norm = torch.sqrt(total)
        factor = s["max_norm"] / norm if norm > s["max_norm"] else torch.ones_like(norm)
        return [norm.view(1), [g.to(f64) * factor for g in s["grads"]]]
    if not c["kind"].endswith("fp4"):
        return _exact_router(c, s)
    if c["kind"] == "product_fp4":
        out = s["out"].to(f64)
        for e, lo, hi in s["spans"]:
            v = torch.mm(s["x"][lo:hi].to(f64), _double(s["w1"][e], s["s1"][e]).mT)
            v = v if s["b1"] is None else v + s["b1"][e].to(f64)
            out[lo:hi] = _activation64(c["act"], v)
            if s["residual"] is not None:
                out[lo:hi] += s["residual"][lo:hi].to(f64)
        return out
    out = torch.zeros(c["T"], c["H"], device="cuda", dtype=f64) if s["residual"] is None else s["residual"].to(f64)
    x = s["x"].to(f64)
    for e in sorted(set(s["idx"].flatten().tolist()) - {-1}):
        share = torch.where(s["idx"] == e, s["w"], torch.zeros_like(s["w"])).to(f64).sum(1)  # this expert's weight in each token
        t = torch.nonzero((s["idx"] == e).any(1))[:, 0]
        v = torch.mm(x[t], _double(s["w1"][e], s["s1"][e]).mT)
        v = v if s["b1"] is None else v + s["b1"][e].to(f64)
        v = torch.mm(_activation64(c["act"], v), _double(s["w2"][e], s["s2"][e]).mT)
        v = v if s["b2"] is None else v + s["b2"][e].to(f64)
        out[t] += share[t, None] * v
    return out
