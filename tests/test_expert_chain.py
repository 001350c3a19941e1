"""The new calls as a user strings them together with the layout, dispatch and
combine: a layer's forward pass by the grouped path and by the few-token call,
and its whole backward pass."""
import pytest
import torch

import product_reference as ref
from test_product import ep, marked, normal  # noqa: F401

pytestmark = pytest.mark.gpu


def layer(T, H, I, E, K, seed):
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand(T, E, generator=g).topk(K, 1).indices.int()
    idx[T // 2, 0] = -1
    tw = torch.softmax(torch.randn(T, K, generator=g), 1)
    x = normal(g, T, H)
    w1, w2 = normal(g, E, 2 * I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    return idx, tw, x, w1, w2, normal(g, T, H)


@pytest.mark.parametrize("T,H,I,E,K,R", [(8, 136, 72, 8, 2, 2), (100, 264, 136, 16, 4, 4), (128, 512, 256, 4, 2, 1)])
def test_forward_paths_agree(ep, T, H, I, E, K, R):  # noqa: F811
    idx, tw, x, w1, w2, res = layer(T, H, I, E, K, T)
    p = ep.Problem.make(T, H, E, K, R, 1, 1, 1)
    p.rank_stride_rows = ep.ep_rank_stride_hint(p)
    bufs = ep.alloc_layout(p)
    d_idx, d_w, d_x, d_w1, d_w2, d_res = (t.cuda() for t in (idx, tw, x, w1, w2, res))
    rows = p.num_rows
    recv, h, y, out = marked(rows, H), marked(rows, I), marked(rows, H), marked(T, H)
    up, down = ep.Product.make(H, I, ep.EP_ACT_SWIGLU), ep.Product.make(I, H)
    seg = (bufs.expert_count, bufs.expert_offset)
    ep.ep_layout_dispatch(p, d_idx, *bufs.args(), None, d_x, d_w, recv, None, None)
    ep.ep_expert_product(p, up, recv, *seg, d_w1, None, None, None, h)
    ep.ep_expert_product(p, down, h, *seg, d_w2, None, None, None, y)
    ep.ep_combine(p, y, bufs.token_slot, d_w, out)
    few = marked(T, H)
    ws = torch.empty(ep.ep_moe_tokens_workspace_bytes(p, up), dtype=torch.uint8, device="cuda")
    ep.ep_moe_tokens(p, up, d_x, d_idx, d_w, d_w1, None, d_w2, None, None, few, ws)
    want, bound = ref.tokens("swiglu", x, idx, tw, w1, None, w2, None, None)
    ref.assert_within(few, want, bound, "few tokens")
    # the grouped path rounds h without its weight (the same relative error)
    # and every expert's row of y to bf16 before the combine
    extra = torch.zeros_like(want)
    for t in range(T):
        for j in range(K):
            e = int(idx[t, j])
            if e >= 0:
                v, err = ref.linear(x[t:t + 1], w1[e], None)
                a = ref.activate("swiglu", v, err)[0]
                row = tw[t, j].double().abs() * (a @ w2[e].double().t()).abs()[0]
                extra[t] += row * ref.HALF_BF16
    ref.assert_within(out, want, bound + 1.01 * extra, "grouped")


def test_backward_chain(ep):  # noqa: F811
    """Gradients of x, the weights and the top-k weights through combine,
    both products and dispatch, against 64-bit autograd of the layer."""
    T, H, I, E, K, R = 60, 136, 72, 4, 2, 2
    idx, tw, x, w1, w2, dout = layer(T, H, I, E, K, 7)
    p = ep.Problem.make(T, H, E, K, R, 1, 1, 1)
    p.rank_stride_rows = ep.ep_rank_stride_hint(p)
    bufs = ep.alloc_layout(p)
    d_idx, d_w, d_x, d_w1, d_w2, d_out = (t.cuda() for t in (idx, tw, x, w1, w2, dout))
    rows, seg = p.num_rows, (bufs.expert_count, bufs.expert_offset)
    up, down = ep.Product.make(H, I, ep.EP_ACT_SWIGLU), ep.Product.make(I, H)
    recv, pre, h, y, out = marked(rows, H), marked(rows, 2 * I), marked(rows, I), marked(rows, H), marked(T, H)
    ep.ep_layout_dispatch(p, d_idx, *bufs.args(), None, d_x, d_w, recv, None, None)
    ep.ep_expert_product(p, up, recv, *seg, d_w1, None, None, pre, h)
    ep.ep_expert_product(p, down, h, *seg, d_w2, None, None, None, y)
    ep.ep_combine(p, y, bufs.token_slot, d_w, out)
    # backward
    dy, dtw = marked(rows, H), torch.empty(T, K, device="cuda")
    ep.ep_combine_backward(p, d_out, y, bufs.token_slot, d_w, dy, dtw)
    dh, dw2 = marked(rows, I), marked(E, H, I)
    ep.ep_expert_product_backward(p, down, dy, None, h, *seg, d_w2, None, dh, dw2)
    dpre, drecv, dw1 = marked(rows, 2 * I), marked(rows, H), marked(E, 2 * I, H)
    ep.ep_expert_product_backward(p, up, dh, pre, recv, *seg, d_w1, dpre, drecv, dw1)
    dx = marked(T, H)
    ep.ep_combine(p, drecv, bufs.token_slot, None, dx)

    X, W1, W2, TW = (t.double().requires_grad_() for t in (x, w1, w2, tw))
    rows_out = []
    for t in range(T):
        o = torch.zeros(H, dtype=torch.float64)
        for j in range(K):
            e = int(idx[t, j])
            if e >= 0:
                g, u = (W1[e] @ X[t]).chunk(2)
                o = o + TW[t, j] * (W2[e] @ (g * torch.sigmoid(g) * u))
        rows_out.append(o)
    (torch.stack(rows_out) * dout.double()).sum().backward()
    # Between the inputs and each gradient lie at most seven roundings to
    # bf16 (pre, h, y, dy, dh, dpre and the gradient's own), each off by 2^-8
    # of its value at most; the errors of the many terms of a sum have either
    # sign, so over a whole gradient the 2-norms keep that relation
    for name, got, want in (("x", dx, X.grad), ("w1", dw1, W1.grad), ("w2", dw2, W2.grad), ("topk_weights", dtw, TW.grad)):
        rel = (got.cpu().double() - want).norm() / want.norm()
        assert rel <= 7 * ref.HALF_BF16, (name, float(rel))
