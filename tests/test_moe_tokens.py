"""The whole expert layer for a few tokens on the GPU against its 64-bit form."""
import pytest
import torch

import product_reference as ref
from test_product import ep, marked, normal  # noqa: F401

pytestmark = pytest.mark.gpu


def route(g, T, E, K, empty=0.0, twice=False):
    idx = torch.rand(T, E, generator=g).topk(K, 1).indices.int() if not twice else torch.randint(0, E, (T, K), generator=g).int()
    idx[torch.rand(T, K, generator=g) < empty] = -1
    return idx


def problem(ep, T, H, E, K):  # noqa: F811
    return ep.Problem.make(T, H, E, K, 1 if E <= 256 else 2, 1, 1, 1)


CASES = [
    # T, H, I, E, K, act, bias, residual, weights, twice, empty
    (1, 8, 8, 1, 1, "none", False, False, False, False, 0.0),
    (1, 264, 136, 16, 4, "swiglu", True, True, True, False, 0.0),
    (3, 72, 200, 4, 2, "geglu", False, True, True, True, 0.2),
    (16, 520, 40, 8, 3, "silu", True, False, True, False, 0.0),
    (17, 136, 264, 5, 5, "gelu", True, True, False, False, 0.1),
    (50, 256, 128, 3, 2, "relu", False, False, True, True, 0.0),
    (90, 328, 72, 64, 8, "swiglu", True, True, True, False, 0.1),
    (128, 64, 64, 2, 2, "swiglu", False, True, True, False, 0.0),
    (128, 40, 24, 300, 32, "geglu", True, True, True, True, 0.1),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])))
def test_tokens(ep, case):  # noqa: F811
    T, H, I, E, K, act, bias, residual, weights, twice, empty = case
    g = torch.Generator().manual_seed(T)
    idx = route(g, T, E, K, empty, twice)
    p, q = problem(ep, T, H, E, K), ep.Product.make(H, I, ref.ACTS.index(act))
    M = q.weight_rows
    x, w1, w2 = normal(g, T, H), normal(g, E, M, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    b1, b2 = (torch.randn(E, M, generator=g), torch.randn(E, H, generator=g)) if bias else (None, None)
    res = normal(g, T, H) if residual else None
    tw = torch.rand(T, K, generator=g) if weights else None
    ws = torch.empty(ep.ep_moe_tokens_workspace_bytes(p, q), dtype=torch.uint8, device="cuda")
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    d = [cuda(t) for t in (x, idx, tw, w1, b1, w2, b2, res)]
    out = marked(T, H)
    ep.ep_moe_tokens(p, q, *d, out, ws)
    assert ep.ep_read_status(ws) == ep.EP_OK
    want, bound = ref.tokens(act, x, idx, tw, w1, b1, w2, b2, res)
    ref.assert_within(out, want, bound)
    # again, into x itself: the same bits
    again = d[0].clone()
    ep.ep_moe_tokens(p, q, again, *d[1:], again, ws)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    if residual:
        again = d[7].clone()
        ep.ep_moe_tokens(p, q, *d[:7], again, again, ws)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16))


FP8_CASES = [
    (1, 128, 128, 4, 2, "swiglu", True),
    (9, 384, 256, 8, 3, "none", False),
    (40, 256, 128, 4, 2, "geglu", True),
    (128, 128, 384, 16, 4, "silu", True),
]


@pytest.mark.parametrize("case", FP8_CASES, ids=lambda c: "-".join(map(str, c[:6])))
def test_tokens_fp8(ep, case):  # noqa: F811
    T, H, I, E, K, act, extras = case
    g = torch.Generator().manual_seed(T)
    idx = route(g, T, E, K, 0.1 if T > 4 else 0.0)
    p, q = problem(ep, T, H, E, K), ep.Product.make(H, I, ref.ACTS.index(act))
    M = q.weight_rows
    x = normal(g, T, H)
    w1, w2 = ((torch.randn(*s, generator=g) * 64).to(torch.float8_e4m3fn) for s in ((E, M, H), (E, H, I)))
    s1 = (torch.rand(E, M // 128, H // 128, generator=g) + 0.5) * (H ** -0.5 / 64)
    s2 = (torch.rand(E, H // 128, I // 128, generator=g) + 0.5) * (I ** -0.5 / 64)
    b1, b2 = (torch.randn(E, M, generator=g), torch.randn(E, H, generator=g)) if extras else (None, None)
    res = normal(g, T, H) if extras else None
    tw = torch.rand(T, K, generator=g)
    ws = torch.empty(ep.ep_moe_tokens_workspace_bytes(p, q), dtype=torch.uint8, device="cuda")
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    out = marked(T, H)
    ep.ep_moe_tokens_fp8(p, q, cuda(x), cuda(idx), cuda(tw), cuda(w1), cuda(s1), cuda(b1), cuda(w2), cuda(s2), cuda(b2),
                         cuda(res), out, ws)
    want, bound = ref.tokens(act, x, idx, tw, w1.float(), b1, w2.float(), b2, res, s1, s2)
    ref.assert_within(out, want, bound)


def small(ep, T=6, E=4, K=2, H=72, I=40):  # noqa: F811
    g = torch.Generator().manual_seed(2)
    p, q = problem(ep, T, H, E, K), ep.Product.make(H, I, ep.EP_ACT_SILU)
    x, w1, w2 = normal(g, T, H).cuda(), normal(g, E, I, H, scale=0.1).cuda(), normal(g, E, H, I, scale=0.1).cuda()
    idx, tw = route(g, T, E, K).cuda(), torch.rand(T, K, generator=g).cuda()
    ws = torch.empty(ep.ep_moe_tokens_workspace_bytes(p, q), dtype=torch.uint8, device="cuda")
    return p, q, x, idx, tw, w1, w2, ws


def test_no_valid_entry_gives_the_residual(ep):  # noqa: F811
    p, q, x, idx, tw, w1, w2, ws = small(ep)
    idx.fill_(-1)
    out = marked(*x.shape)
    ep.ep_moe_tokens(p, q, x, idx, tw, w1, None, w2, None, None, out, ws)
    assert not out.any()
    ep.ep_moe_tokens(p, q, x, idx, tw, w1, None, w2, None, x, out, ws)
    assert torch.equal(out, x)


def test_no_tokens(ep):  # noqa: F811
    p, q, x, idx, tw, w1, w2, ws = small(ep)
    p.num_tokens = 0
    ws.fill_(255)
    out = marked(1, 72)
    ep.ep_moe_tokens(p, q, x, idx, tw, w1, None, w2, None, None, out, ws)
    assert ep.ep_read_status(ws) == ep.EP_OK and (out.view(torch.int16) == 0x7A51).all()


def test_bad_ids_count_as_empty_and_are_reported(ep):  # noqa: F811
    p, q, x, idx, tw, w1, w2, ws = small(ep)
    want, out = marked(*x.shape), marked(*x.shape)
    idx[2, 1] = -1
    ep.ep_moe_tokens(p, q, x, idx, tw, w1, None, w2, None, None, want, ws)
    assert ep.ep_read_status(ws) == ep.EP_OK
    for bad in (4, -2, 2 ** 31 - 1, -2 ** 31):
        idx[2, 1] = bad
        ep.ep_moe_tokens(p, q, x, idx, tw, w1, None, w2, None, None, out, ws)
        assert ep.ep_read_status(ws) == ep.EP_ERR_BAD_EXPERT
        assert torch.equal(out, want)
    idx[2, 1] = -1
    ep.ep_moe_tokens(p, q, x, idx, tw, w1, None, w2, None, None, out, ws)
    assert ep.ep_read_status(ws) == ep.EP_OK


def test_values_that_are_not_finite_stay_with_their_tokens(ep):  # noqa: F811
    """A token's NaN and an expert's infinite weights reach only that token and those that name the expert."""
    p, q, x, idx, tw, w1, w2, ws = small(ep, T=40, E=8)
    clean, out = marked(*x.shape), marked(*x.shape)
    ep.ep_moe_tokens(p, q, x, idx, tw, w1, None, w2, None, None, clean, ws)
    x[5, 3] = float("nan")
    w1[6, 2] = float("inf")
    w2[6] = float("nan")
    ep.ep_moe_tokens(p, q, x, idx, tw, w1, None, w2, None, None, out, ws)
    hit = (idx == 6).any(1)
    hit[5] = True
    assert torch.isnan(out[hit]).all() and 0 < int(hit.sum()) < 40
    assert torch.equal(out[~hit], clean[~hit])


def test_graph_replays(ep):  # noqa: F811
    """Replays follow the routing that the captured buffers hold, and two graphs with workspaces of their own mix."""
    p, q, x, idx, tw, w1, w2, ws = small(ep, T=20, E=8)
    ids = [idx.clone(), idx.flip(0).contiguous()]
    want = []
    for i in ids:
        o = marked(*x.shape)
        ep.ep_moe_tokens(p, q, x, i, tw, w1, None, w2, None, x, o, ws)
        want.append(o)
    torch.cuda.synchronize()
    outs, graphs, spaces = [marked(*x.shape) for _ in range(2)], [], [ws, ws.clone()]
    for o, s in zip(outs, spaces):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            ep.ep_moe_tokens(p, q, x, idx, tw, w1, None, w2, None, x, o, s)
    for n in range(4):
        idx.copy_(ids[n % 2])
        for o, gr in zip(outs, graphs):
            o.zero_()
            gr.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, want[n % 2])
