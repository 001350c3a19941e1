"""The experts' products, their gradients and the few-token layer at the ends
of what the header allows: dense calls of every kind, the most experts, the
widest features, the largest weight, and a problem whose batch is not the one
that the arrays hold."""
import pytest
import torch

import product_reference as ref
from test_moe_tokens import route
from test_product import Routed, ep, marked, normal, untouched  # noqa: F401

pytestmark = pytest.mark.gpu


def backward(ep, p, q, arrays, dout, pre, x, w):  # noqa: F811
    """dpre, dx, dweight and dbias of one call, in marked buffers."""
    rows, M, E = x.shape[0], q.weight_rows, p.num_experts
    dpre = None if pre is None else marked(rows, M)
    dx, dw, db = marked(rows, q.in_features), marked(E, M, q.in_features), torch.full((E, M), 7.0, device="cuda")
    ws = torch.empty(ep.ep_product_workspace_bytes(p, q), dtype=torch.uint8, device="cuda")
    cuda = [None if t is None else t.cuda() for t in (dout, pre, x)]
    ep.ep_expert_product_backward(p, q, *cuda, *arrays, w.cuda(), dpre, dx, dw, None, db, ws)
    return dpre, dx, dw, db


def check_backward(act, got, rows, e, dout, pre, x, w):
    want = ref.backward(act, dout[rows], dout[rows] if pre is None else pre[rows], x[rows], w[e])
    dpre, dx, dw, db = got
    if pre is not None:
        ref.assert_within(dpre[rows], *want["dpre"], f"dpre of expert {e}")
    ref.assert_within(dx[rows], *want["dx"], f"dx of expert {e}")
    ref.assert_within(dw[e], *want["dweight"], f"dweight of expert {e}")
    ref.assert_within(db[e], *want["dbias"], f"dbias of expert {e}")


@pytest.mark.parametrize("T,C,N,act", [(1, 72, 40, "none"), (37, 264, 136, "swiglu"), (1000, 136, 200, "gelu")])
def test_dense_backward(ep, T, C, N, act):  # noqa: F811
    p, q = ep.Problem.make(T, 8, 1, 1, 1, 1, 1, T + 5), ep.Product.make(C, N, ref.ACTS.index(act))
    g = torch.Generator().manual_seed(T)
    x, w, dout = normal(g, T, C), normal(g, 1, q.weight_rows, C, scale=C ** -0.5), normal(g, T, N)
    pre = None if act == "none" else normal(g, T, q.weight_rows)
    check_backward(act, backward(ep, p, q, (None, None), dout, pre, x, w), slice(0, T), 0, dout, pre, x, w)


@pytest.mark.parametrize("T,C,N", [(1, 256, 128), (37, 384, 256), (400, 128, 384)])
def test_dense_fp8(ep, T, C, N):  # noqa: F811
    p, q = ep.Problem.make(T, 8, 1, 1, 1, 1, 1, T), ep.Product.make(C, N, ep.EP_ACT_GEGLU)
    g = torch.Generator().manual_seed(T)
    x, w = ((torch.randn(*s, generator=g) * 64).to(torch.float8_e4m3fn) for s in ((T, C), (2 * N, C)))
    xs, ws = torch.rand(T, C // 128, generator=g) / 64, torch.rand(2 * N // 128, C // 128, generator=g) / 512
    out = marked(T + 2, N)
    ep.ep_expert_product_fp8(p, q, x.cuda(), xs.cuda(), C // 128, 1, None, None, w.cuda(), ws.cuda(), None, None, out)
    o, b, _, _ = ref.product("geglu", x.float(), w.float(), scales=(xs, ws))
    ref.assert_within(out[:T], o, b)
    assert untouched(out, list(range(T)))


@pytest.mark.parametrize("T,K", [(64, 2), (3000, 8)])
def test_most_experts(ep, T, K):  # noqa: F811
    """2048 experts, many of them without rows, on 8 ranks."""
    E, C, N = ep.EP_MAX_EXPERTS, 40, 24
    r = Routed(ep, T, E, K, R=8, empty=0.1, seed=T)
    q, g = ep.Product.make(C, N, ep.EP_ACT_SWIGLU), torch.Generator().manual_seed(T)
    x, w, dout = normal(g, r.rows, C), normal(g, E, 2 * N, C, scale=C ** -0.5), normal(g, r.rows, N)
    out, pre = marked(r.rows, N), marked(r.rows, 2 * N)
    ep.ep_expert_product(r.p, q, x.cuda(), *r.arrays, w.cuda(), None, None, pre, out)
    assert untouched(out, r.used) and untouched(pre, r.used)
    got = [t.cpu() for t in backward(ep, r.p, q, r.arrays, dout, pre, x, w)]
    out, pre = out.cpu(), pre.cpu()
    for e, rows in r.of.items():
        if rows:
            o, b, v, vb = ref.product("swiglu", x[rows], w[e])
            ref.assert_within(out[rows], o, b, f"out of expert {e}")
            ref.assert_within(pre[rows], v, vb, f"pre of expert {e}")
            check_backward("swiglu", got, rows, e, dout, pre, x, w)
        else:
            assert not got[2][e].any() and not got[3][e].any()


def test_most_entries_of_the_few_token_layer(ep):  # noqa: F811
    """128 tokens, top-32 of 2048 experts, some named twice."""
    T, K, E, H, I = ep.EP_MOE_TOKENS_MAX, ep.EP_MAX_TOPK, ep.EP_MAX_EXPERTS, 40, 24
    g = torch.Generator().manual_seed(0)
    idx = route(g, T, E, K, 0.05, True)
    idx[:, 1] = idx[:, 0]
    p, q = ep.Problem.make(T, H, E, K, 8, 1, 1, 1), ep.Product.make(H, I, ep.EP_ACT_SILU)
    x, w1, w2 = normal(g, T, H), normal(g, E, I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    b1, b2, tw = torch.randn(E, I, generator=g), torch.randn(E, H, generator=g), torch.rand(T, K, generator=g)
    ws, out = torch.empty(ep.ep_moe_tokens_workspace_bytes(p, q), dtype=torch.uint8, device="cuda"), marked(T, H)
    ep.ep_moe_tokens(p, q, x.cuda(), idx.cuda(), tw.cuda(), w1.cuda(), b1.cuda(), w2.cuda(), b2.cuda(), None, out, ws)
    assert ep.ep_read_status(ws) == ep.EP_OK
    ref.assert_within(out, *ref.tokens("silu", x, idx, tw, w1, b1, w2, b2, None))


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("C,N", [(1 << 16, 8), (8, 1 << 16), (1 << 16, 264)])
def test_widest_products(ep, T, C, N):  # noqa: F811
    r = Routed(ep, T, 2, 1, seed=T)
    act = "swiglu" if N == 8 or C == 8 else "silu"
    q, g = ep.Product.make(C, N, ref.ACTS.index(act)), torch.Generator().manual_seed(T)
    x, w, dout = normal(g, r.rows, C), normal(g, 2, q.weight_rows, C, scale=C ** -0.5), normal(g, r.rows, N)
    out, pre = marked(r.rows, N), marked(r.rows, q.weight_rows)
    ep.ep_expert_product(r.p, q, x.cuda(), *r.arrays, w.cuda(), None, None, pre, out)
    pre = pre.cpu()
    got = backward(ep, r.p, q, r.arrays, dout, pre, x, w)
    for e, rows in r.of.items():
        o, b, v, vb = ref.product(act, x[rows], w[e])
        ref.assert_within(out[rows], o, b, f"out of expert {e}")
        ref.assert_within(pre[rows], v, vb, f"pre of expert {e}")
        check_backward(act, got, rows, e, dout, pre, x, w)


@pytest.mark.parametrize("H,I", [(1 << 16, 8), (8, 1 << 16)])
def test_widest_few_token_layers(ep, H, I):  # noqa: F811
    T, E, K = 5, 4, 2
    g = torch.Generator().manual_seed(0)
    idx = route(g, T, E, K)
    p, q = ep.Problem.make(T, H, E, K, 1, 1, 1, 1), ep.Product.make(H, I, ep.EP_ACT_SWIGLU)
    x, w1, w2 = normal(g, T, H), normal(g, E, 2 * I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    ws, out = torch.empty(ep.ep_moe_tokens_workspace_bytes(p, q), dtype=torch.uint8, device="cuda"), marked(T, H)
    ep.ep_moe_tokens(p, q, x.cuda(), idx.cuda(), None, w1.cuda(), None, w2.cuda(), None, None, out, ws)
    ref.assert_within(out, *ref.tokens("swiglu", x, idx, None, w1, None, w2, None, None))


@pytest.mark.parametrize("T", [5, 40])
def test_largest_weight(ep, T):  # noqa: F811
    """2^31 values, 4 GiB: outputs and gradients of rows at both ends of the
    weight and about its middle, where byte offsets pass 2^31."""
    C, M = 1 << 15, 1 << 16
    p, q = ep.Problem.make(T, 8, 1, 1, 1, 1, 1, T), ep.Product.make(C, M)
    g = torch.Generator().manual_seed(T)
    x, few = normal(g, T, C), normal(g, 1, 48, C, scale=C ** -0.5)
    at = torch.cat([torch.arange(16), torch.arange(M // 2 - 8, M // 2 + 8), torch.arange(M - 16, M)])
    w = torch.zeros(M, C, dtype=torch.bfloat16, device="cuda")
    w[at.cuda()] = few[0].cuda()
    out = marked(T, M)
    ep.ep_expert_product(p, q, x.cuda(), None, None, w, None, None, None, out)
    o, b, _, _ = ref.product("none", x, few[0])
    ref.assert_within(out[:, at.cuda()], o, b, "out")
    assert int((out != 0).sum()) <= T * 48
    # dx sums over all rows of the weight, all but 48 of them zeros
    dout, some = torch.zeros(T, M, dtype=torch.bfloat16, device="cuda"), normal(g, T, 48)
    dout[:, at.cuda()] = some.cuda()
    dx, dw = marked(T, C), marked(M, C)
    ep.ep_expert_product_backward(p, q, dout, None, x.cuda(), None, None, w, None, dx, dw)
    want = ref.backward("none", some, some, x, few[0])
    # the zeros are added as well: a longer sum of the same magnitudes
    v, bound = want["dx"]
    bound = bound + (some.double().abs() @ few[0].double().abs()) * (M * ref.ULP32)
    ref.assert_within(dx, v, bound, "dx")
    ref.assert_within(dw[at.cuda()], *want["dweight"], "dweight")
    assert int((dw != 0).any(1).sum()) <= 48


@pytest.mark.parametrize("tokens", [1, 16384])
def test_batch_is_a_hint(ep, tokens):  # noqa: F811
    """The rows are the arrays'; a problem of another batch gives the same results."""
    E, C, N = 4, 136, 72
    r = Routed(ep, 300, E, 2, R=2, seed=1)
    q, g = ep.Product.make(C, N, ep.EP_ACT_SILU), torch.Generator().manual_seed(1)
    x, w, dout = normal(g, r.rows, C), normal(g, E, N, C, scale=C ** -0.5), normal(g, r.rows, N)
    other = ep.Problem.make(tokens, 8, E, 1, 2, 1, 1, r.p.rank_stride_rows)
    out, pre = marked(r.rows, N), marked(r.rows, N)
    ep.ep_expert_product(other, q, x.cuda(), *r.arrays, w.cuda(), None, None, pre, out)
    assert untouched(out, r.used)
    pre = pre.cpu()
    got = backward(ep, other, q, r.arrays, dout, pre, x, w)
    assert untouched(got[1], r.used)
    for e, rows in r.of.items():
        o, b, v, vb = ref.product("silu", x[rows], w[e])
        ref.assert_within(out[rows], o, b, f"out of expert {e}")
        ref.assert_within(pre[rows], v, vb, f"pre of expert {e}")
        check_backward("silu", got, rows, e, dout, pre, x, w)
