"""The router, the 4-bit layer and the clipping as a user strings them together with what stands between them: a
training step from logits to clipped gradients, and a decode step on 4-bit weights."""
import math

import pytest
import torch

import fp4_reference as fp4
import product_reference as ref
import route_reference as rref
from test_grads import check
from test_product import ep, marked, normal  # noqa: F401

pytestmark = pytest.mark.gpu


def test_training_step(ep):  # noqa: F811
    """Logits by a dense product, the router with its losses, the layer, and back to the router's weight and the
    tokens; then the clipping of all weights' gradients.  Against 64-bit autograd with the choices held."""
    T, H, I, E, K, R = 60, 136, 72, 8, 2, 2
    g = torch.Generator().manual_seed(7)
    x, wg = normal(g, T, H), normal(g, E, H, scale=H ** -0.5)
    w1, w2 = normal(g, E, 2 * I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    dout, coeff = normal(g, T, H), torch.tensor([3.0, 0.2])
    mask = torch.ones(T, dtype=torch.uint8)
    mask[5] = mask[59] = 0
    d = lambda t: t.cuda()  # noqa: E731
    p = ep.Problem.make(T, H, E, K, R, 1, 1, 1)
    p.rank_stride_rows = ep.ep_rank_stride_hint(p)
    one, gate = ep.Problem.make(T, H, 1, 1, 1, 1, 1, T), ep.Product.make(H, E)
    router = ep.Router.make(ep.EP_SCORE_SOFTMAX, True, 1.0, True)
    bufs = ep.alloc_layout(p)
    rows, seg = p.num_rows, (bufs.expert_count, bufs.expert_offset)
    up, down = ep.Product.make(H, I, ep.EP_ACT_SWIGLU), ep.Product.make(I, H)

    logits = marked(T, E)
    ep.ep_expert_product(one, gate, d(x), None, None, d(wg), None, None, None, logits)
    idx, tw = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    count, tokens = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    prob, losses = torch.empty(E, device="cuda"), torch.empty(2, device="cuda")
    ws = torch.empty(ep.ep_route_workspace_bytes(p, router), dtype=torch.uint8, device="cuda")
    ep.ep_route(p, router, logits, None, d(mask), idx, tw, count, tokens, prob, losses, ws)
    recv, pre, h, y, out = marked(rows, H), marked(rows, 2 * I), marked(rows, I), marked(rows, H), marked(T, H)
    ep.ep_layout_dispatch(p, idx, *bufs.args(), None, d(x), tw, recv, None, None)
    assert torch.equal(bufs.expert_count, count)  # the layout counts what the router counted
    ep.ep_expert_product(p, up, recv, *seg, d(w1), None, None, pre, h)
    ep.ep_expert_product(p, down, h, *seg, d(w2), None, None, None, y)
    ep.ep_combine(p, y, bufs.token_slot, tw, out)

    dy, dtw = marked(rows, H), torch.empty(T, K, device="cuda")
    ep.ep_combine_backward(p, d(dout), y, bufs.token_slot, tw, dy, dtw)
    dh, dw2 = marked(rows, I), marked(E, H, I)
    ep.ep_expert_product_backward(p, down, dy, None, h, *seg, d(w2), None, dh, dw2)
    dpre, drecv, dw1 = marked(rows, 2 * I), marked(rows, H), marked(E, 2 * I, H)
    ep.ep_expert_product_backward(p, up, dh, pre, recv, *seg, d(w1), dpre, drecv, dw1)
    dx = marked(T, H)
    ep.ep_combine(p, drecv, bufs.token_slot, None, dx)
    dlogits = marked(T, E)
    ep.ep_route_backward(p, router, logits, idx, d(mask), count, tokens, dtw, d(coeff), dlogits)
    dx_gate, dwg = marked(T, H), marked(E, H)
    ep.ep_expert_product_backward(one, gate, dlogits, None, d(x), None, None, d(wg), None, dx_gate, dwg)
    grads = [dwg, dw1, dw2]
    before = [t.clone() for t in grads]
    square, norm = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda")
    held = ep.Grads.make(grads)
    gws = torch.empty(ep.ep_grad_workspace_bytes(held), dtype=torch.uint8, device="cuda")
    ep.ep_grad_square_sum(held, square, gws)
    ep.ep_grad_clip(held, square, 1.0, norm)
    check(grads, grads, before, float(norm), float(square), 1.0)

    # each step against its own formula, on what the step before left
    lo, i, n = logits.cpu(), idx.cpu(), int(tokens)
    assert torch.equal(i, rref.choose(0, lo, None, mask, K)) and n == T - 2
    want = rref.statistics(0, lo, i, mask, K)
    ref.assert_within(losses, *want["losses"], "losses")
    value, bound = rref.gradient(0, True, 1.0, lo, i, mask, count.cpu(), n, dtw.cpu(), coeff, K, True)
    ref.assert_within(dlogits, value, bound, "dlogits")
    back = ref.backward("none", dlogits.cpu(), None, x, wg)
    ref.assert_within(before[0], *back["dweight"], "router's weight")
    ref.assert_within(dx_gate, *back["dx"], "tokens through the router")

    # and the whole: 64-bit autograd from the tokens, with the choices and counts held
    X, WG, W1, W2 = (t.double().requires_grad_() for t in (x, wg, w1, w2))
    v = X @ WG.t()
    total = rref.objective(0, True, 1.0, v[mask != 0], i[mask != 0], None, count.cpu(), n, None, coeff, K)
    c = torch.softmax(v.gather(1, i.long().clamp_min(0)), -1)
    rows_out = []
    for t in range(T):
        o = torch.zeros(H, dtype=torch.float64)
        for j in range(K):
            if i[t, j] >= 0:
                a, b = (W1[int(i[t, j])] @ X[t]).chunk(2)
                o = o + c[t, j] * (W2[int(i[t, j])] @ (a * torch.sigmoid(a) * b))
        rows_out.append(o)
    (total + (torch.stack(rows_out) * dout.double()).sum()).backward()
    # Between the inputs and a gradient lie at most nine roundings to bf16 (the logits, pre, h, y, dy, dh, dpre or
    # dlogits, the gradient's own, and the sum of the tokens' two), each off by 2^-8 of its value at most; a logit's
    # error moves a weight by as much as its size, here up to 4.  Errors of a sum's terms have either sign, so the
    # 2-norms keep that relation.
    bound = (9 + 4) * ref.HALF_BF16
    for name, got, exact in (("x", dx.double() + dx_gate.double(), X.grad), ("router", before[0], WG.grad),
                             ("w1", before[1], W1.grad), ("w2", before[2], W2.grad)):
        rel = (got.cpu().double() - exact).norm() / exact.norm()
        assert rel <= bound, (name, float(rel))
    exact = math.sqrt(sum(float((t.grad ** 2).sum()) for t in (WG, W1, W2)))
    assert abs(float(norm) - exact) <= bound * exact


@pytest.mark.parametrize("T", [1, 20, 128])
def test_decode_step_on_4_bit_weights(ep, T):  # noqa: F811
    """A shared expert by the dense product, whose result is the residual of the routed ones that the router names."""
    H, I, E, K = 160, 96, 12, 3
    g = torch.Generator().manual_seed(T)
    x, wg = normal(g, T, H), normal(g, E, H, scale=H ** -0.5)
    make = lambda *s: fp4.quantise(torch.randn(*s, generator=g) * s[-1] ** -0.5)  # noqa: E731
    w1, w2, shared1, shared2 = make(E, 2 * I, H), make(E, H, I), make(1, 2 * I, H), make(1, H, I)
    bias = torch.randn(E, generator=g) * 0.1
    d = lambda t: t.cuda()  # noqa: E731
    p = ep.Problem.make(T, H, E, K, 1, 1, 1, 1)
    dense = ep.Problem.make(T, H, 1, 1, 1, 1, 1, T)
    up, down = ep.Product.make(H, I, ep.EP_ACT_SWIGLU), ep.Product.make(I, H)
    router = ep.Router.make(ep.EP_SCORE_SIGMOID, True, 2.5, False)
    logits = (x.double() @ wg.double().t()).float()
    idx, tw = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    hidden, res, out = marked(T, I), marked(T, H), marked(T, H)
    ws = torch.empty(ep.ep_moe_tokens_workspace_bytes(p, up), dtype=torch.uint8, device="cuda")
    ep.ep_route(p, router, d(logits), d(bias), None, idx, tw)
    ep.ep_expert_product_fp4(dense, up, d(x), None, None, *map(d, shared1), None, None, hidden)
    ep.ep_expert_product_fp4(dense, down, hidden, None, None, *map(d, shared2), None, None, res)
    ep.ep_moe_tokens_fp4(p, up, d(x), idx, tw, *map(d, w1), None, *map(d, w2), None, res, out, ws)
    assert ep.ep_read_status(ws) == ep.EP_OK
    want = rref.choose(1, logits, bias, None, K)
    assert torch.equal(idx.cpu(), want)
    ref.assert_within(tw, *rref.weights(1, True, 2.5, logits, want))
    o, bound, _, _ = ref.product("swiglu", x, fp4.values(*shared1)[0])
    ref.assert_within(hidden, o, bound)
    o, bound, _, _ = ref.product("none", hidden.cpu(), fp4.values(*shared2)[0])
    ref.assert_within(res, o, bound)
    o, bound = ref.tokens("swiglu", x, want, tw.cpu(), fp4.values(*w1), None, fp4.values(*w2), None, res.cpu())
    ref.assert_within(out, o, bound)
