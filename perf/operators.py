"""Workloads of the expert products, the few-token expert layer and the combine's gradient.

``run`` computes a workload's operator either with plain torch operations in 32 bits
(``own = False``) or with the library's entry points (``own = True``).  Sizes follow the
routing workloads of ``ep_inputs.py`` (hidden 7168 or 4096, top-8 of 64 to 256 experts, 128 to
16384 tokens); the experts' inner width is 2048, or an uneven 1400 or 1408.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu", "swiglu", "geglu")  # in the order of the EP_ACT_* codes

DEFAULTS = dict(T=1, H=256, I=256, E=1, K=1, R=1, act="none", bias=False, residual=False, zipf=0.0, empty=0.0)


def _case(kind, name=None, **kw):
    c = {"kind": kind, **DEFAULTS, **kw}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # a shared expert's down projection on a small batch: one dense product, with the residual stream added
        _case("product", "dense-37-residual", T=37, H=2048, I=7168, bias=True, residual=True),
        # ragged experts of uneven width: Zipf popularity, some padded tokens, bias
        _case("product", "zipf-1000-geglu", T=1000, H=4096, I=1400, E=128, K=8, R=8, act="geglu", bias=True, zipf=1.2,
              empty=0.05),
        # the up projection of a long prefill over all experts, gated
        _case("product", "experts-16384-swiglu", T=16384, H=7168, I=2048, E=256, K=8, R=16, act="swiglu"),
        # a decode batch's up projection on FP8-dispatched rows: the weights are the traffic
        _case("product_fp8", "fp8-100-swiglu", T=100, H=4096, I=1408, E=128, K=8, act="swiglu"),
        # a prefill's up projection on FP8-dispatched rows
        _case("product_fp8", "fp8-4096-swiglu", T=4096, H=7168, I=2048, E=256, K=8, R=8, act="swiglu"),
        # a fine-tuning step's experts on a short ragged batch, with biases
        _case("backward", "backward-1000-geglu", T=1000, H=2048, I=1400, E=32, K=4, R=4, act="geglu", bias=True, zipf=1.2),
        # a training step's up projection
        _case("backward", "backward-16384-swiglu", T=16384, H=7168, I=2048, E=64, K=8, R=8, act="swiglu"),
        # one token being generated
        _case("tokens", "tokens-1-swiglu", T=1, H=7168, I=2048, E=64, K=8, act="swiglu", residual=True),
        # the decode batch: nearly every expert is reached by a few tokens
        _case("tokens", "tokens-128-swiglu", T=128, H=7168, I=2048, E=256, K=8, act="swiglu"),
        # a small batch on FP8 weights, one token of it padding
        _case("tokens_fp8", "tokens-fp8-17-swiglu", T=17, H=4096, I=1408, E=128, K=8, act="swiglu", bias=True, residual=True,
              empty=0.06),
        # gradient of the combine of a decode-sized and of a large batch
        _case("combine", "combine-128", T=128, H=7168, E=256, K=8, R=8),
        _case("combine", "combine-16384", T=16384, H=7168, E=256, K=8, R=16),
    ]


def _spread(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high + 1)))
    return max(low, min(high, int(v))) // step * step


def draw(rng):
    kind = rng.choice(("product", "product", "product_fp8", "backward", "tokens", "tokens_fp8", "combine"))
    fp8 = kind.endswith("fp8")
    while True:
        dense = kind in ("product", "backward") and rng.random() < 0.25
        E = 1 if dense else 2 ** rng.randint(2, 8)
        K = 1 if dense else rng.randint(1, min(8, E))
        c = _case(
            kind, E=E, K=K, R=1 if dense else 2 ** rng.randint(0, 2),
            T=_spread(rng, 1, 128 if kind.startswith("tokens") else 16384),
            H=_spread(rng, 128, 7168, 128 if fp8 else 8), I=_spread(rng, 128, 4096, 128 if fp8 else 8),
            act=rng.choice(ACTS), bias=rng.random() < 0.5, residual=kind != "backward" and rng.random() < 0.5,
            zipf=rng.choice((0.0, 0.0, 1.2)), empty=0.0 if dense else rng.choice((0.0, 0.0, 0.1)))
        flops = work(c)["flops"]
        weights = E * _width(c) * c["H"]
        if kind == "combine" or (flops <= 4e12 and weights <= 2e9):
            return c


def _width(c):
    """Rows of an expert's weight: both halves of a gated activation."""
    return c["I"] * (2 if c["act"] in ("swiglu", "geglu") else 1)


def work(c):
    T, H, I, K, E = c["T"], c["H"], c["I"], c["K"], c["E"]
    M = _width(c)
    rows = T * K * (1 - c["empty"])
    touched = E * (1 - (1 - min(1.0, K / E)) ** T)  # experts that a uniform router reaches
    el = 1 if c["kind"].endswith("fp8") else 2
    if c["kind"] in ("product", "product_fp8"):
        by = rows * H * el + rows * I * 2 * (2 if c["residual"] else 1) + touched * M * H * el
        return {"bytes": int(by), "flops": int(2 * rows * M * H)}
    if c["kind"] == "backward":
        pre = 0 if c["act"] == "none" else M
        by = rows * (I + pre + 2 * H) * 2 + 2 * E * M * H * 2
        return {"bytes": int(by), "flops": int(4 * rows * M * H)}
    if c["kind"] in ("tokens", "tokens_fp8"):
        by = touched * (M * H + H * I) * el + T * H * 2 * (3 if c["residual"] else 2)
        return {"bytes": int(by), "flops": int(2 * rows * (M * H + H * I))}
    return {"bytes": int(T * H * 2 + 2 * rows * H * 2), "flops": int(3 * rows * H)}


def _routing(c, g):
    """What a router and the layout leave: ids and weights, each expert's rows, and each entry's row."""
    T, E, K, R = c["T"], c["E"], c["K"], c["R"]
    logits = torch.randn(T, E, device="cuda", generator=g)
    if c["zipf"]:  # popularity (e+1)^-s: Gumbel noise on its logarithm
        rank = torch.arange(1, E + 1, device="cuda", dtype=torch.float32)
        logits = -c["zipf"] * rank.log() - (-torch.rand(T, E, device="cuda", generator=g).clamp_min(1e-20).log()).log()
    top = logits.topk(K, 1)
    idx, w = top.indices.int(), torch.softmax(top.values.float(), 1)
    if c["empty"]:  # padded tokens name no expert
        idx[torch.rand(T, device="cuda", generator=g) < c["empty"]] = -1
    idx, w = idx.contiguous(), w.contiguous()
    flat = idx.flatten().long()
    count = torch.bincount(flat[flat >= 0], minlength=E)
    first = count.cumsum(0) - count
    L = E // R
    offset = first - first[::L].repeat_interleave(L)  # inside the rank's slice
    # the capacity of a slice: the worst case where that is little, else a margin over the mean; rows past it are dropped
    S = T * K if R == 1 else min(T * min(K, L), (4 if c["zipf"] else 5 / 4) * T * K // R + 64)
    S = int(S)
    base = torch.arange(E, device="cuda") // L * S + offset
    order = flat.argsort(stable=True)
    slot = torch.full((T * K,), -1, device="cuda", dtype=torch.int32)
    valid = order[flat[order] >= 0]
    e = flat[valid]
    at = torch.arange(valid.numel(), device="cuda") - first[e]
    slot[valid] = torch.where(offset[e] + at < S, base[e] + at, -1).int()
    held = torch.minimum(count, (S - offset).clamp_min(0))
    spans = [(i, b, b + n) for i, (b, n) in enumerate(zip(base.tolist(), held.tolist())) if n]
    return {"idx": idx, "w": w, "count": count.int(), "offset": offset.int().contiguous(), "slot": slot.view(T, K),
            "spans": spans, "S": S, "rows": R * S}


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    t = torch.randn(*shape, device="cuda", generator=g, dtype=dtype)
    return t.mul_(scale) if scale != 1.0 else t


def _codes(g, *shape):
    """e4m3 codes of normal values that fill the type's range, and one scale for 128 x 128 (weights) or 1 x 128 (rows)."""
    return _normal(g, *shape, scale=64.0).to(torch.float8_e4m3fn)


def _scales(g, *shape, scale):
    return (torch.rand(*shape, device="cuda", generator=g) + 0.5) * scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, H, I, E, K = c["T"], c["H"], c["I"], c["E"], c["K"]
    M = _width(c)
    s = {"case": c, **_routing(c, g)}
    rows = s["rows"]
    bf = dict(device="cuda", dtype=torch.bfloat16)
    if c["kind"] in ("product", "product_fp8"):
        if c["kind"] == "product":
            s["x"] = _normal(g, rows, H)
            s["weight"] = _normal(g, E, M, H, scale=H ** -0.5)
        else:
            s["x"], s["x_sf"] = _codes(g, rows, H), _scales(g, rows, H // 128, scale=1 / 64)
            s["weight"] = _codes(g, E, M, H)
            s["w_sf"] = _scales(g, E, M // 128, H // 128, scale=H ** -0.5 / 64)
        s["bias"] = _normal(g, E, M, dtype=torch.float32) if c["bias"] else None
        s["residual"] = _normal(g, rows, I) if c["residual"] else None
        s["out"] = torch.zeros(rows, I, **bf)
    elif c["kind"] == "backward":
        s["x"] = _normal(g, rows, H)
        s["weight"] = _normal(g, E, M, H, scale=H ** -0.5)
        s["dout"] = _normal(g, rows, I)
        s["pre"] = None if c["act"] == "none" else _normal(g, rows, M)
        s["dpre"] = None if c["act"] == "none" else torch.zeros(rows, M, **bf)
        s["dx"] = torch.zeros(rows, H, **bf)
        s["dweight"] = torch.empty(E, M, H, **bf)
        s["dbias"] = torch.empty(E, M, device="cuda") if c["bias"] else None
    elif c["kind"] in ("tokens", "tokens_fp8"):
        s["x"] = _normal(g, T, H)
        if c["kind"] == "tokens":
            s["w1"] = _normal(g, E, M, H, scale=H ** -0.5)
            s["w2"] = _normal(g, E, H, I, scale=I ** -0.5)
        else:
            s["w1"], s["w2"] = _codes(g, E, M, H), _codes(g, E, H, I)
            s["w1_sf"] = _scales(g, E, M // 128, H // 128, scale=H ** -0.5 / 64)
            s["w2_sf"] = _scales(g, E, H // 128, I // 128, scale=I ** -0.5 / 64)
        s["b1"] = _normal(g, E, M, dtype=torch.float32) if c["bias"] else None
        s["b2"] = _normal(g, E, H, dtype=torch.float32) if c["bias"] else None
        s["residual"] = _normal(g, T, H) if c["residual"] else None
        s["out"] = torch.empty(T, H, **bf)
    else:
        s["dout"], s["y"] = _normal(g, T, H), _normal(g, rows, H)
        s["dy"] = torch.zeros(rows, H, **bf)
        s["dweights"] = torch.empty(T, K, device="cuda")
    return s


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


def _act_grad(name, v, d):
    """The gradient of the pre-activations `v`, from that of the activation's output `d`."""
    if name == "none":
        return d
    if name == "relu":
        return d * (v > 0)
    if name in ("swiglu", "geglu"):
        a, b = v.chunk(2, -1)
        one = "silu" if name == "swiglu" else "gelu"
        return torch.cat([_act_grad(one, a, d * b), d * _act(one, a)], -1)
    if name == "silu":
        sg = torch.sigmoid(v)
        return d * (sg * (1 + v * (1 - sg)))
    return d * (0.5 * (1 + torch.erf(v * 0.5 ** 0.5)) + v * torch.exp(-0.5 * v * v) * (2 * math.pi) ** -0.5)


def _wide(t, sf, up):
    """The values of e4m3 codes `t` with one scale for each 128 columns and `up` rows."""
    sf = sf.repeat_interleave(128, -1)
    return t.float() * (sf.repeat_interleave(up, -2) if up > 1 else sf)


def _plain_product(s):
    c = s["case"]
    for e, lo, hi in s["spans"]:
        if c["kind"] == "product":
            v = s["x"][lo:hi].float() @ s["weight"][e].float().t()
        else:
            v = _wide(s["x"][lo:hi], s["x_sf"][lo:hi], 1) @ _wide(s["weight"][e], s["w_sf"][e], 128).t()
        if s["bias"] is not None:
            v = v + s["bias"][e]
        v = _act(c["act"], v)
        if s["residual"] is not None:
            v = v + s["residual"][lo:hi].float()
        s["out"][lo:hi] = v.bfloat16()
    return s["out"]


def _plain_backward(s):
    c = s["case"]
    s["dweight"].zero_()
    if s["dbias"] is not None:
        s["dbias"].zero_()
    for e, lo, hi in s["spans"]:
        d = s["dout"][lo:hi].float()
        d = d if s["pre"] is None else _act_grad(c["act"], s["pre"][lo:hi].float(), d)
        s["dx"][lo:hi] = (d @ s["weight"][e].float()).bfloat16()
        s["dweight"][e] = (d.t() @ s["x"][lo:hi].float()).bfloat16()
        if s["dbias"] is not None:
            s["dbias"][e] = d.sum(0)
    return [s["dx"], s["dweight"], s["dbias"]]


def _plain_tokens(s):
    c = s["case"]
    acc = torch.zeros_like(s["x"], dtype=torch.float32) if s["residual"] is None else s["residual"].float()
    for e in s["idx"].unique().tolist():
        if e < 0:
            continue
        t, j = (s["idx"] == e).nonzero(as_tuple=True)
        if c["kind"] == "tokens":
            w1, w2 = s["w1"][e].float(), s["w2"][e].float()
        else:
            w1, w2 = _wide(s["w1"][e], s["w1_sf"][e], 128), _wide(s["w2"][e], s["w2_sf"][e], 128)
        v = s["x"][t].float() @ w1.t()
        if s["b1"] is not None:
            v = v + s["b1"][e]
        v = _act(c["act"], v) @ w2.t()
        if s["b2"] is not None:
            v = v + s["b2"][e]
        acc[t] += v * s["w"][t, j, None]  # a router names an expert once for a token
    return acc.bfloat16()


def _plain_combine(s):
    slot = s["slot"].long()
    hit = slot >= 0
    d = s["dout"].float()
    y = s["y"][slot.clamp_min(0)].float()
    s["dweights"].copy_((d[:, None] * y).sum(-1) * hit)
    t, j = hit.nonzero(as_tuple=True)
    s["dy"][slot[t, j]] = (d[t] * s["w"][t, j, None]).bfloat16()
    return [s["dy"], s["dweights"]]


def _own(s):
    import combine_ep_get_amd as ep

    c = s["case"]
    kind = c["kind"]
    p = ep.Problem.make(c["T"], c["H"], c["E"], c["K"], c["R"], 1, 1, s["S"])
    if kind == "combine":
        ep.ep_combine_backward(p, s["dout"], s["y"], s["slot"], s["w"], s["dy"], s["dweights"])
        return [s["dy"], s["dweights"]]
    q = ep.Product.make(c["H"], c["I"], ACTS.index(c["act"]))
    if kind == "product":
        ep.ep_expert_product(p, q, s["x"], s["count"], s["offset"], s["weight"], s["bias"], s["residual"], None, s["out"])
        return s["out"]
    if kind == "product_fp8":
        ep.ep_expert_product_fp8(p, q, s["x"], s["x_sf"], c["H"] // 128, 1, s["count"], s["offset"], s["weight"], s["w_sf"],
                                 s["bias"], s["residual"], s["out"])
        return s["out"]
    if kind == "backward":
        if "workspace" not in s:
            s["workspace"] = torch.empty(ep.ep_product_workspace_bytes(p, q), device="cuda", dtype=torch.uint8)
        ep.ep_expert_product_backward(p, q, s["dout"], s["pre"], s["x"], s["count"], s["offset"], s["weight"], s["dpre"],
                                      s["dx"], s["dweight"], None, s["dbias"], s["workspace"])
        return [s["dx"], s["dweight"], s["dbias"]]
    if "workspace" not in s:
        s["workspace"] = torch.empty(ep.ep_moe_tokens_workspace_bytes(p, q), device="cuda", dtype=torch.uint8)
    if kind == "tokens":
        ep.ep_moe_tokens(p, q, s["x"], s["idx"], s["w"], s["w1"], s["b1"], s["w2"], s["b2"], s["residual"], s["out"],
                         s["workspace"])
    else:
        ep.ep_moe_tokens_fp8(p, q, s["x"], s["idx"], s["w"], s["w1"], s["w1_sf"], s["b1"], s["w2"], s["w2_sf"], s["b2"],
                             s["residual"], s["out"], s["workspace"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind in ("product", "product_fp8"):
        return _plain_product(state)
    if kind == "backward":
        return _plain_backward(state)
    return _plain_combine(state) if kind == "combine" else _plain_tokens(state)


def _double(codes, sf, block_rows):
    """float64 values of codes with scales: rows in blocks of `block_rows`, columns in blocks of 128."""
    R, C = codes.shape
    v = codes.to(torch.float64).view(R // block_rows, block_rows, C // 128, 128)
    return (v * sf.double()[:, None, :, None]).view(R, C)


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
    fp8 = c["kind"].endswith("fp8")
    if c["kind"] == "combine":
        dy, dw = s["dy"].to(torch.float64), torch.zeros(c["T"], c["K"], device="cuda", dtype=f64)
        d = s["dout"].to(f64)
        for j in range(c["K"]):
            at = s["slot"][:, j].long()
            t = torch.nonzero(at >= 0)[:, 0]
            dy[at[t]] = s["w"][t, j].to(f64).unsqueeze(1) * d[t]
            dw[t, j] = torch.linalg.vecdot(d[t], s["y"][at[t]].to(f64))
        return [dy, dw]
    if c["kind"].startswith("product"):
        out = s["out"].to(f64)
        for e, lo, hi in s["spans"]:
            if fp8:
                v = torch.mm(_double(s["x"][lo:hi], s["x_sf"][lo:hi], 1), _double(s["weight"][e], s["w_sf"][e], 128).mT)
            else:
                v = torch.mm(s["x"][lo:hi].to(f64), s["weight"][e].to(f64).mT)
            v = v if s["bias"] is None else v + s["bias"][e].to(f64)
            out[lo:hi] = _activation64(c["act"], v)
        used = torch.zeros(s["rows"], 1, device="cuda", dtype=f64)
        for _, lo, hi in s["spans"]:
            used[lo:hi] = 1
        return out if s["residual"] is None else out + used * s["residual"].to(f64)
    if c["kind"] == "backward":
        dx = s["dx"].to(f64)
        dweight = torch.zeros(s["dweight"].shape, device="cuda", dtype=f64)
        dbias = None if s["dbias"] is None else torch.zeros(s["dbias"].shape, device="cuda", dtype=f64)
        for e, lo, hi in s["spans"]:
            d = s["dout"][lo:hi].to(f64)
            if s["pre"] is not None:  # the derivative by differentiation, not by its formula
                with torch.enable_grad():
                    v = s["pre"][lo:hi].to(f64).requires_grad_()
                    d, = torch.autograd.grad(_activation64(c["act"], v), v, d)
            dx[lo:hi] = torch.mm(d, s["weight"][e].to(f64))
            dweight[e] = torch.mm(d.mT, s["x"][lo:hi].to(f64))
            if dbias is not None:
                dbias[e] = d.sum(0)
        return [dx, dweight, dbias]
    out = torch.zeros(c["T"], c["H"], device="cuda", dtype=f64) if s["residual"] is None else s["residual"].to(f64)
    x = s["x"].to(f64)
    for e in sorted(set(s["idx"].flatten().tolist()) - {-1}):
        share = torch.where(s["idx"] == e, s["w"], torch.zeros_like(s["w"])).to(f64).sum(1)  # this expert's weight in each token
        t = torch.nonzero((s["idx"] == e).any(1))[:, 0]
        w1 = _double(s["w1"][e], s["w1_sf"][e], 128) if fp8 else s["w1"][e].to(f64)
        w2 = _double(s["w2"][e], s["w2_sf"][e], 128) if fp8 else s["w2"][e].to(f64)
        v = torch.mm(x[t], w1.mT)
        v = v if s["b1"] is None else v + s["b1"][e].to(f64)
        v = torch.mm(_activation64(c["act"], v), w2.mT)
        v = v if s["b2"] is None else v + s["b2"][e].to(f64)
        out[t] += share[t, None] * v
    return out
