"""Plain 64-bit forms of the experts' products, the few-token layer and the
combine's gradient, each with a bound on how far fp32 sums and the stated
roundings can be off.  Independent of the library; runs on the CPU.

Bounds.  A sum of n fp32 products off by at most an ulp (2^-23) a step is
within n * 2^-23 * sum|terms| of the exact one.  A matrix instruction on e4m3
operands aligns the products of a block to the largest before it adds them:
2^-12 of a block's sum|terms| bounds what that drops (8.7e-5 = 2^-13.5 was seen
on codes of all magnitudes).  Rounding to bf16 is off by 2^-8 of the value
at most (half a step), and by half the smallest subnormal."""
import math

import torch

F64 = torch.float64
ULP32 = 2.0 ** -23
HALF_BF16 = 2.0 ** -8
FP8_BLOCK = 2.0 ** -12
TINY = 2.0 ** -133  # half of bf16's smallest subnormal is 2^-134
ACTS = ("none", "relu", "gelu", "silu", "swiglu", "geglu")  # by EP_ACT_* code
# largest slope of each activation's first input: gelu 1.129, silu 1.0999
SLOPE = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "silu": 1.1}
# exp2, reciprocal and erfc in fp32: relative error of the factor beside v
ACT_EVAL = 2.0 ** -19


def gated(act):
    return act in ("swiglu", "geglu")


def one(act, v):
    act = {"swiglu": "silu", "geglu": "gelu"}.get(act, act)
    if act == "none":
        return v
    if act == "relu":
        return v.clamp_min(0)
    return v / (1 + torch.exp(-v)) if act == "silu" else 0.5 * v * torch.special.erfc(-v / math.sqrt(2))


def slope_name(act):
    return {"swiglu": "silu", "geglu": "gelu"}.get(act, act)


def activate(act, v, err):
    """act(v) and its bound, for v known within err."""
    s = SLOPE[slope_name(act)]
    if not gated(act):
        a = one(act, v)
        return a, s * err + ACT_EVAL * v.abs()
    g, u = v.chunk(2, -1)
    eg, eu = err.chunk(2, -1)
    a = one(act, g)
    ea = s * eg + ACT_EVAL * g.abs()
    return a * u, ea * (u.abs() + eu) + a.abs() * eu + 2.0 ** -22 * (a * u).abs()


def rounded(v, err):
    """Bound after one rounding to bf16 of a value known within err."""
    return err + HALF_BF16 * (v.abs() + err) + TINY


def linear(x, w, b, *, scales=None):
    """x w^T + b for one expert and its bound.  scales: (x_sf, w_sf) of e4m3 codes."""
    x, w = x.to(F64), w.to(F64)
    if scales is not None:
        xs, ws = scales
        x = x * xs.to(F64).repeat_interleave(128, -1)
        w = w * ws.to(F64).repeat_interleave(128, -1).repeat_interleave(128, -2)
    v, mag = x @ w.t(), x.abs() @ w.abs().t()
    n = x.shape[-1] + 8
    if b is not None:
        v, mag = v + b.to(F64), mag + b.to(F64).abs()
    return v, mag * (n * ULP32 + (FP8_BLOCK if scales is not None else 0.0))


def product(act, x, w, b=None, residual=None, scales=None):
    """(out, bound, pre, pre bound) of the rows of one expert."""
    v, err = linear(x, w, b, scales=scales)
    o, oerr = activate(act, v, err)
    if residual is not None:
        o = o + residual.to(F64)
        oerr = oerr + ULP32 * o.abs()
    return o, rounded(o, oerr), v, rounded(v, err)


def act_grad(act, pre, dout):
    """dpre by differentiation in 64 bits."""
    if act == "none":
        return dout.to(F64)
    v = pre.to(F64).requires_grad_()
    if gated(act):
        g, u = v.chunk(2, -1)
        o = one(act, g) * u
    else:
        o = one(act, v)
    return torch.autograd.grad(o, v, dout.to(F64))[0]


def backward(act, dout, pre, x, w):
    """{name: (value, bound)} of dpre, dx, dweight and dbias of one expert's rows."""
    d = act_grad(act, pre, dout)
    # slopes are of order 1 and cancel: their fp32 evaluation is off by a few
    # ulp of the terms, at most 2 (|v| + 1) each
    size = dout.to(F64).abs()
    if act == "none":
        derr = torch.zeros_like(d)
    elif gated(act):
        g, u = pre.to(F64).abs().chunk(2, -1)
        derr = torch.cat([size * u * 2 * (g + 1), size * 2 * (g + 1)], -1) * ACT_EVAL
    else:
        derr = size * 2 * (pre.to(F64).abs() + 1) * ACT_EVAL
    dr = derr if act == "none" else rounded(d, derr)  # dout itself is not rounded again
    x, w = x.to(F64), w.to(F64)
    dx, dxe = d @ w, dr @ w.abs() + (d.abs() @ w.abs()) * ((d.shape[-1] + 8) * ULP32)
    dw, dwe = d.t() @ x, dr.t() @ x.abs() + (d.abs().t() @ x.abs()) * ((d.shape[0] + 8) * ULP32)
    db, dbe = d.sum(0), derr.sum(0) + d.abs().sum(0) * ((d.shape[0] + 8) * ULP32)
    return {"dpre": (d, rounded(d, derr)), "dx": (dx, rounded(dx, dxe)), "dweight": (dw, rounded(dw, dwe)),
            "dweight_acc": (dw, dwe), "dbias": (db, dbe)}


def tokens(act, x, idx, weights, w1, b1, w2, b2, residual, s1=None, s2=None):
    """out and bound of the few-token layer.  s1, s2: scales of e4m3 weights."""
    T, K = idx.shape
    E = w1.shape[0]
    out = torch.zeros(T, w2.shape[1], dtype=F64) if residual is None else residual.to(F64).clone()
    err = torch.zeros_like(out)
    mag = out.abs()
    terms = 8
    for t in range(T):
        for j in range(K):
            e = int(idx[t, j])
            if not 0 <= e < E:
                continue
            wt = 1.0 if weights is None else float(weights[t, j])
            a, b = w1[e].to(F64), w2[e].to(F64)
            if s1 is not None:
                a = a * s1[e].to(F64).repeat_interleave(128, -1).repeat_interleave(128, -2)
                b = b * s2[e].to(F64).repeat_interleave(128, -1).repeat_interleave(128, -2)
            v, verr = linear(x[t:t + 1], a, None if b1 is None else b1[e])
            h, herr = activate(act, v, verr)
            hr = rounded(wt * h, abs(wt) * (herr + 2 * K * ULP32 * h.abs()))
            y = (wt * h) @ b.t()
            err[t] += (hr @ b.abs().t())[0]
            mag[t] += ((wt * h).abs() @ b.abs().t())[0]
            if b2 is not None:
                y = y + wt * b2[e].to(F64)
                mag[t] += abs(wt) * b2[e].to(F64).abs()
            out[t] += y[0]
            terms += b.shape[1] + 2
    # every term of every expert of a token may be added in turn
    n = K * (w2.shape[2] + 2) + 16
    return out, rounded(out, err + mag * (n * ULP32))


def combine_backward(dout, y, slot, weights, rows):
    """dy as {row: (value, bound)} stacked in slot order, and dweights with its bound."""
    T, K = slot.shape
    d = dout.to(F64)
    ok = (slot >= 0) & (slot < rows)
    at = slot.clamp(0, rows - 1).long()
    w = torch.ones(T, K, dtype=F64) if weights is None else weights.to(F64)
    dy = w[..., None] * d[:, None]
    yy = y.to(F64)[at]
    dw = (d[:, None] * yy).sum(-1)
    mag = (d[:, None] * yy).abs().sum(-1)
    zero = torch.zeros_like(dw)
    return ok, dy, rounded(dy, ULP32 * dy.abs()), torch.where(ok, dw, zero), torch.where(ok, mag * ((d.shape[1] + 8) * ULP32), zero)


def assert_within(got, want, bound, what=""):
    got = got.detach().cpu().to(F64)
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        worst = ((got - want).abs() / bound.clamp_min(1e-300))[bad].nan_to_num(math.inf).max()
        first = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values outside the bound, the worst "
                             f"{float(worst):.3g} times it, the first at {first}: got "
                             f"{float(got[tuple(first)])}, want {float(want[tuple(first)])}")


def layout(idx, E, R, S, A=1):
    """Rows of every expert and every entry's row, by the layout's definition: {e: [rows]}, slot [T,K]."""
    T, K = idx.shape
    L = E // R
    counts = [0] * E
    for t in range(T):
        for j in range(K):
            e = int(idx[t, j])
            if 0 <= e < E:
                counts[e] += 1
    offset, base = [0] * E, 0
    for e in range(E):
        base = 0 if e % L == 0 else base
        offset[e] = base
        base += (counts[e] + A - 1) // A * A
    rows = {e: [] for e in range(E)}
    slot = torch.full((T, K), -1, dtype=torch.int32)
    for t in range(T):
        for j in range(K):
            e = int(idx[t, j])
            if not 0 <= e < E:
                continue
            at = offset[e] + len(rows[e])
            inside = at < S
            rows[e].append(e // L * S + at if inside else -1)
            if inside:
                slot[t, j] = rows[e][-1]
    return {e: [r for r in v if r >= 0] for e, v in rows.items()}, slot, counts, offset
