"""Plain 64-bit forms of the router, its balance loss and its gradient, each
with a bound on how far fp32 arithmetic can be off.  Independent of the library;
runs on the CPU.

Bounds.  An exponential of a difference d of two logits is off by |d| / 2 ulp
(the difference's rounding) and one ulp of its own, in ulps of 2^-23; a sum over
n experts by at most 40 roundings (up to 32 values of a lane, then 6 steps), a
division by one: REL(D) = (48 + D) 2^-23 of its value bounds a score, a
probability or a weight, D being the largest |d| of the row.  A sum over T
tokens adds at most T + 16 roundings; terms of a difference are bounded by
the sum of their sizes."""
import math

import torch

F64 = torch.float64
ULP32 = 2.0 ** -23
HALF_BF16 = 2.0 ** -8
SOFTMAX, SIGMOID = 0, 1


def softmax(v):
    e = torch.exp(v - v.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def scores(kind, v):
    """Scores and the probabilities of the balance loss, of rows with some logit above -inf."""
    if kind == SOFTMAX:
        s = softmax(v)
        return s, s
    # numerators that a row of very small logits does not take to 0
    top = v.amax(-1, keepdim=True).clamp_max(0)
    num = torch.where(v < 0, torch.exp(v - top), torch.exp(-top)) / (1 + torch.exp(-v.abs()))
    return 1 / (1 + torch.exp(-v)), num / num.sum(-1, keepdim=True)


def spread(v):
    """D of every row: over its finite logits, and from 0."""
    f = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    return f.abs().amax(-1, keepdim=True) * 2


def live_rows(logits, mask):
    v = logits.to(F64)
    ok = torch.isnan(v).any(-1) | (v > -math.inf).any(-1)
    return ok if mask is None else ok & (mask != 0)


def choose(kind, logits, bias, mask, K):
    """idx [T,K] by sorting exact keys."""
    v = logits.to(F64)
    T, E = v.shape
    ok = torch.ones(T, dtype=torch.bool) if mask is None else mask != 0
    if bias is None:
        key = v.clone()
    else:
        safe = torch.where(ok[:, None], v, torch.zeros_like(v))
        if kind == SOFTMAX:
            safe = torch.where((safe > -math.inf).any(-1, keepdim=True), safe, torch.zeros_like(safe))
            s = softmax(safe)
        else:
            s = 1 / (1 + torch.exp(-safe))
        key = torch.where(v > -math.inf, s + bias.to(F64), torch.full_like(v, -math.inf))
    key = torch.where(torch.isnan(key) | torch.isnan(v), torch.full_like(key, -math.inf), key)
    key[~ok] = -math.inf
    top, at = torch.sort(key, dim=-1, descending=True, stable=True)
    if K > E:
        top = torch.cat([top, torch.full((T, K - E), -math.inf, dtype=F64)], 1)
        at = torch.cat([at, torch.zeros(T, K - E, dtype=at.dtype)], 1)
    return torch.where(top[:, :K] > -math.inf, at[:, :K], -1).int()


def weights(kind, normalise, scale, logits, idx):
    """w [T,K] and its bound for choices idx (rows of finite or -inf logits)."""
    v = logits.to(F64)
    hit = (idx >= 0) & (idx < v.shape[1])
    some = hit.any(-1, keepdim=True)
    safe = torch.where(some, v, torch.zeros_like(v))
    at = idx.long().clamp(0, v.shape[1] - 1)
    if normalise:
        # over the chosen ones; numerators as in scores
        c = torch.where(hit, safe.gather(1, at), torch.full(at.shape, -math.inf, dtype=F64))
        c = torch.where(some, c, torch.zeros_like(c))
        u = softmax(c) if kind == SOFTMAX else scores(SIGMOID, c)[1]
    else:
        u = scores(kind, safe)[0].gather(1, at)
    w = torch.where(hit, u * scale, torch.zeros_like(u))
    return w, w.abs() * (48 + spread(safe)) * ULP32 + 1e-37


def statistics(kind, logits, idx, mask, K):
    """{name: (value, bound)} of the counts, V, the probabilities' sums and both losses."""
    v = logits.to(F64)
    T, E = v.shape
    live = live_rows(logits, mask)
    v, ids = v[live], idx[live].flatten().long()
    ids = ids[(ids >= 0) & (ids < E)]
    count = torch.bincount(ids, minlength=E)
    V = v.shape[0]
    if V == 0:
        z = torch.zeros(E, dtype=F64)
        return {"expert_count": (count, 0), "token_count": (V, 0), "prob_sum": (z, z), "losses": (z.new_zeros(2), z.new_zeros(2))}
    p = scores(kind, v)[1]
    D = spread(v)
    prob = p.sum(0)
    perr = (p * (48 + D)).sum(0) * ULP32 + prob * (T + 16) * ULP32
    scale = E / (K * V * V)
    lse = torch.logsumexp(v, -1)
    lerr = ((48 + D[:, 0]) + lse.abs() + 2) * ULP32
    losses = torch.stack([scale * (count * prob).sum(), (lse ** 2).sum() / V])
    bound = torch.stack([scale * (count * perr).sum(), (2 * lse.abs() * lerr + lerr ** 2).sum() / V]) + losses * 4 * ULP32
    return {"expert_count": (count, 0), "token_count": (V, 0), "prob_sum": (prob, perr), "losses": (losses, bound)}


def objective(kind, normalise, scale, v, idx, live, count, V, dweights, dlosses, K):
    """sum dweights w + dlosses . losses as a function of the live rows' logits, counts and choices held."""
    E = v.shape[1]
    s, p = scores(kind, v)
    total = v.new_zeros(())
    if dlosses is not None:
        total = total + dlosses[0].to(F64) * E / (K * V * V) * (count.to(F64) * p.sum(0)).sum()
        total = total + dlosses[1].to(F64) / V * (torch.logsumexp(v, -1) ** 2).sum()
    if dweights is not None:
        hit = (idx >= 0) & (idx < E)
        at = idx.long().clamp(0, E - 1)
        u = torch.where(hit, s.gather(1, at), torch.zeros(at.shape, dtype=F64))
        if normalise and kind == SOFTMAX:  # the softmax of the chosen logits: the others' derivative is 0 and not a rounding
            some = hit.any(-1, keepdim=True)
            c = torch.where(hit | ~some, v.gather(1, at), torch.full(at.shape, -math.inf, dtype=F64))
            u = torch.where(hit, softmax(c), torch.zeros(at.shape, dtype=F64))
        elif normalise:
            u = u / u.sum(-1, keepdim=True).clamp_min(1e-300)
        total = total + (torch.where(hit, dweights.to(F64), torch.zeros_like(u)) * u).sum() * scale
    return total


def gradient(kind, normalise, scale, logits, idx, mask, count, V, dweights, dlosses, K, out_bf16):
    """dlogits and its bound: by differentiation, bounded by the sizes of the terms."""
    T, E = logits.shape
    live = live_rows(logits, mask)
    out, bound = torch.zeros(T, E, dtype=F64), torch.zeros(T, E, dtype=F64)
    if not live.any():
        return out, bound
    v = logits[live].to(F64).requires_grad_()
    i = None if idx is None else idx[live]
    dw = None if dweights is None else dweights[live]
    n = max(1, int(V))
    d, = torch.autograd.grad(objective(kind, normalise, scale, v, i, live, count, n, dw, dlosses, K), v)
    v = v.detach()
    s, p = scores(kind, v)
    size = torch.zeros_like(v)
    if dlosses is not None:
        b = dlosses[0].to(F64).abs() * E / (K * n * n) * (count.to(F64) - K * n / E).abs()
        size += p * (b + (p * b).sum(-1, keepdim=True))
        size += dlosses[1].to(F64).abs() * 2 / n * torch.logsumexp(v, -1, keepdim=True).abs() * softmax(v)
        # logsumexp itself is off by ulps of its terms, not of their sum
        size += dlosses[1].to(F64).abs() * 2 / n * softmax(v)
    if dw is not None:
        hit = (i >= 0) & (i < E)
        at = i.long().clamp(0, E - 1)
        u = torch.where(hit, s.gather(1, at), torch.zeros(at.shape, dtype=F64))
        if normalise:
            u = u / u.sum(-1, keepdim=True).clamp_min(1e-300)
        g = torch.where(hit, dw.to(F64).abs() * abs(scale), torch.zeros_like(u))
        each = u * (g + (u * g).sum(-1, keepdim=True))
        size.scatter_add_(1, at, torch.where(hit, each, torch.zeros_like(each)))
        if not normalise and kind == SOFTMAX:
            size += s * (g * u).sum(-1, keepdim=True)
    err = 4 * size * (48 + spread(v)) * ULP32 + 1e-37
    if out_bf16:
        err = err + HALF_BF16 * (d.abs() + err) + 2.0 ** -133
    out[live], bound[live] = d, err
    return out, bound
