"""Host-side refusals of the router, the gradients' clipping and the 4-bit products: nothing is enqueued, so no GPU
is needed.  And the 64-bit forms that the GPU tests compare with, against plain torch."""
import ctypes
import math

import pytest
import torch

import combine_ep_get_amd as ep
import fp4_reference as fp4
import route_reference as ref
from test_product_abi import A, BAD, P, Q, call


def R(score=0, normalise=1, bf16=0, scale=1.0):
    return ep.Router(score, normalise, bf16, scale)


def route(p=None, r=None, logits=A, bias=A, mask=A, idx=A, w=A, count=A, tokens=A, prob=A, losses=A, ws=A, n=1 << 30):
    return call("ep_route", p or P(), r or R(), logits, bias, mask, idx, w, count, tokens, prob, losses, ws, n, None)


def balance(p=None, r=None, logits=A, idx=A, mask=A, count=A, tokens=A, prob=A, losses=A, ws=A, n=1 << 30):
    return call("ep_balance_loss", p or P(), r or R(), logits, idx, mask, count, tokens, prob, losses, ws, n, None)


def backward(p=None, r=None, logits=A, idx=A, mask=A, count=A, tokens=A, dw=A, dl=A, out=A):
    return call("ep_route_backward", p or P(), r or R(), logits, idx, mask, count, tokens, dw, dl, out, None)


ALL = (route, balance, backward)
STATS = ("count", "tokens", "prob", "losses")


@pytest.mark.parametrize("fn", ALL, ids=lambda f: f.__name__)
def test_bad_problems_and_routers(fn):
    for bad in (dict(E=9), dict(K=0), dict(K=33), dict(H=250), dict(T=-1), dict(E=4096, R=16)):
        assert fn(p=P(**bad)) == BAD, bad
    for bad in (R(score=-1), R(score=2), R(normalise=2), R(normalise=-1), R(bf16=2), R(scale=math.inf), R(scale=math.nan)):
        assert fn(r=bad) == BAD
    assert ep.load().ep_route_workspace_bytes(ctypes.byref(P()), None) == 0


def test_pointers():
    for fn, names in ((route, "logits idx w ws"), (balance, "logits idx ws"), (backward, "logits idx count tokens out")):
        for name in names.split():
            assert fn(**{name: None}) == BAD, (fn.__name__, name)
        assert fn(logits=A + 8) == BAD
    assert backward(out=A + 8) == BAD
    for name in STATS:  # all or none
        assert route(**{name: None}) == BAD and balance(**{name: None}) == BAD
        assert route(**{name: A + 2}) == BAD and balance(**{name: A + 2}) == BAD
    for name in ("bias", "idx", "w"):
        assert route(**{name: A + 2}) == BAD
    for name in ("idx", "count", "tokens", "dw", "dl"):
        assert backward(**{name: A + 2}) == BAD
    need = ep.ep_route_workspace_bytes(P(), R())
    assert need > 0
    for fn in (route, balance):
        assert fn(n=need - 1) == BAD and fn(ws=A + 128) == BAD
    none = dict(count=None, tokens=None, prob=None, losses=None, ws=None, n=0)
    assert route(p=P(T=0), logits=None, idx=None, w=None, **none) == ep.EP_OK  # nothing to do, and no statistics
    assert balance(**none) == BAD
    assert backward(p=P(T=0), logits=None, out=None, idx=None) == ep.EP_OK


def test_the_slice_stride_is_not_needed():
    assert ep.ep_route_workspace_bytes(P(S=0), R()) > 0
    assert ep.ep_route_workspace_bytes(P(T=1 << 26, K=1), R()) <= 256 + 512 * (12 + 8 * 8)


def grads(*items):
    return (ep.Grad * len(items))(*[ep.Grad(*i) for i in items])


def test_gradient_lists():
    lib = ep.load()

    def both(array, n, sq=A, ws=A, nbytes=1 << 30, max_norm=1.0):
        return (lib.ep_grad_square_sum(array, n, sq, ws, nbytes, None), lib.ep_grad_clip(array, n, sq, max_norm, A, None))

    ok = (A, A, 10, 0, 0)
    for bad in ((A, A, -1, 0, 0), (A, A, 1 << 40, 0, 0), (A, A, 10, 2, 0), (A, A, 10, -1, 0), (A, A, 10, 0, 1),
                (None, A, 10, 0, 0), (A + 1, A, 10, 0, 0), (A + 2, A, 10, 1, 0)):
        array = grads(ok, bad)
        assert both(array, 2) == (BAD, BAD), bad
        assert ep.load().ep_grad_workspace_bytes(array, 2) == 0
    for bad in ((A, None, 10, 0, 0), (A, A + 1, 10, 0, 0), (A, A + 2, 10, 1, 0)):  # where it goes
        assert lib.ep_grad_clip(grads(bad), 1, A, 1.0, A, None) == BAD
    assert both(None, 1) == (BAD, BAD) and both(grads(ok), -1) == (BAD, BAD)
    assert both(grads(ok), 1, sq=A + 4) == (BAD, BAD) and both(grads(ok), 1, sq=None) == (BAD, BAD)
    for max_norm in (-1.0, math.nan):
        assert lib.ep_grad_clip(grads(ok), 1, A, max_norm, A, None) == BAD
    assert lib.ep_grad_clip(grads(ok), 1, A, 1.0, A + 2, None) == BAD
    need = lib.ep_grad_workspace_bytes(grads(ok), 1)
    assert need > 0 and lib.ep_grad_workspace_bytes(None, 0) > 0
    assert lib.ep_grad_square_sum(grads(ok), 1, A, A, need - 1, None) == BAD
    assert lib.ep_grad_square_sum(grads(ok), 1, A, A + 8, need, None) == BAD
    assert lib.ep_grad_square_sum(grads(ok), 1, A, None, need, None) == BAD


def test_gradient_binding():
    with pytest.raises(ValueError, match="gradient 0: a cpu tensor"):
        ep.Grads.make([torch.zeros(3)])
    with pytest.raises(ValueError, match="dtype torch.float16"):
        ep.Grads.make([torch.zeros(3, dtype=torch.float16)])
    with pytest.raises(ValueError, match="dtype torch.float32 into torch.bfloat16"):
        ep.Grads.make([torch.zeros(3)], [torch.zeros(3, dtype=torch.bfloat16)])
    with pytest.raises(ValueError, match="out 0|outs: tensor 0 has 4"):
        ep.Grads.make([torch.zeros(3)], [torch.zeros(4)])
    with pytest.raises(ValueError, match="2 tensors for 1"):
        ep.Grads.make([torch.zeros(3)], [torch.zeros(3), torch.zeros(3)])
    with pytest.raises(ValueError, match="contiguous"):
        ep.Grads.make([torch.zeros(4, 4).t()])
    assert len(ep.Grads.make([])) == 0


def product_fp4(p=None, q=None, x=A, count=A, offset=A, w=A, sf=A, bias=A, res=A, out=A):
    return call("ep_expert_product_fp4", p or P(), q or Q(), x, count, offset, w, sf, bias, res, out, None)


def tokens_fp4(p=None, q=None, x=A, idx=A, tw=A, w1=A, s1=A, b1=A, w2=A, s2=A, b2=A, res=A, out=A, ws=A, n=1 << 30):
    return call("ep_moe_tokens_fp4", p or P(), q or Q(), x, idx, tw, w1, s1, b1, w2, s2, b2, res, out, ws, n, None)


def test_fp4_refusals():
    for fn in (product_fp4, tokens_fp4):
        for bad in (dict(E=9), dict(K=0), dict(T=-1), dict(T=ep.EP_MOE_TOKENS_MAX + 1)):
            assert fn(p=P(**bad)) == BAD, bad
        for bad in (Q(C=264), Q(N=136), Q(C=16), Q(act=6), Q(reserved=1), Q(N=(1 << 16) + 32)):
            assert fn(q=bad, p=P(H=max(8, bad.in_features))) == BAD, (bad.in_features, bad.out_features)
    for fn, names, bad in ((product_fp4, "x w sf bias res out", A + 8), (product_fp4, "x w sf out count offset", None),
                           (tokens_fp4, "x w1 s1 b1 w2 s2 b2 res out", A + 8), (tokens_fp4, "x idx w1 s1 w2 s2 out ws", None)):
        for name in names.split():
            assert fn(**{name: bad}) == BAD, (fn.__name__, name, bad)
    assert tokens_fp4(q=Q(C=288), p=P(H=256)) == BAD
    assert ep.load().ep_expert_product_fp4(None, ctypes.byref(Q()), A, A, A, A, A, A, A, A, None) == BAD
    dense = dict(count=None, offset=None)
    assert product_fp4(**dense) == BAD
    assert product_fp4(p=P(T=0)) == ep.EP_OK


def test_binding_checks():
    p, q, r = P(), Q(), R()
    with pytest.raises(ValueError, match="w_sf: .* the call uses 16384"):
        ep.ep_expert_product_fp4(p, q, A, A, A, A, torch.zeros(16383, dtype=torch.uint8), None, None, A, stream=0)
    with pytest.raises(ValueError, match="w_fp4: .* the call uses 262144"):
        ep.ep_expert_product_fp4(p, q, A, A, A, torch.zeros(262143, dtype=torch.uint8), A, None, None, A, stream=0)
    with pytest.raises(ValueError, match="w2_sf: dtype"):
        ep.ep_moe_tokens_fp4(p, q, A, A, A, A, A, None, A, torch.zeros(9), None, None, A, A, 1 << 30, stream=0)
    with pytest.raises(ValueError, match="logits: dtype torch.bfloat16"):
        ep.ep_route(p, r, torch.zeros(64, 8, dtype=torch.bfloat16), None, None, A, A, stream=0)
    with pytest.raises(ValueError, match="logits: 511 elements"):
        ep.ep_route(p, r, torch.zeros(511), None, None, A, A, stream=0)
    with pytest.raises(ValueError, match="token_mask: 63 elements"):
        ep.ep_balance_loss(p, r, A, A, torch.zeros(63, dtype=torch.uint8), A, A, A, A, A, 1 << 30, stream=0)
    with pytest.raises(ValueError, match="losses: 1 elements"):
        ep.ep_route(p, r, A, None, None, A, A, A, A, A, torch.zeros(1), A, 1 << 30, stream=0)
    with pytest.raises(ValueError, match="dlogits: dtype"):
        ep.ep_route_backward(p, r, A, A, None, A, A, A, A, torch.zeros(64, 8, dtype=torch.bfloat16), stream=0)
    with pytest.raises(ep.EpError, match="invalid argument"):
        ep.ep_route(p, R(score=5), A, None, None, A, A, stream=0)


@pytest.mark.parametrize("kind", [0, 1])
def test_reference_scores_match_torch(kind):
    g = torch.Generator().manual_seed(1)
    v = torch.randn(20, 33, generator=g, dtype=torch.float64) * 3
    s, p = ref.scores(kind, v)
    plain = torch.softmax(v, -1) if kind == 0 else torch.sigmoid(v)
    assert torch.allclose(s, plain, rtol=1e-13) and torch.allclose(p, plain / plain.sum(-1, keepdim=True), rtol=1e-13)
    idx = ref.choose(kind, v, None, None, 5)
    assert torch.equal(idx.long(), v.topk(5, -1).indices)
    w, _ = ref.weights(kind, True, 2.0, v, idx)
    want = plain.gather(1, idx.long())
    assert torch.allclose(w, 2 * want / want.sum(-1, keepdim=True), rtol=1e-13)


def test_reference_balance_is_one_for_even_choices():
    v = torch.zeros(12, 6)
    idx = torch.arange(24).view(12, 2) % 6
    st = ref.statistics(0, v, idx, None, 2)
    assert abs(float(st["losses"][0][0]) - 1) < 1e-12 and abs(float(st["losses"][0][1]) - math.log(6) ** 2) < 1e-12


def test_reference_sees_a_mistake():
    """A weight off by a thousandth, a gradient without one of its terms or of the neighbouring row is outside the bound."""
    from product_reference import assert_within
    g = torch.Generator().manual_seed(2)
    v = torch.randn(10, 16, generator=g)
    idx = ref.choose(0, v, None, None, 3)
    w, bound = ref.weights(0, True, 1.0, v, idx)
    assert_within(w.float(), w, bound)
    st = ref.statistics(0, v, idx, None, 3)
    dw, dl = torch.randn(10, 3, generator=g), torch.tensor([1.0, 1.0])
    full, gb = ref.gradient(0, True, 1.0, v, idx, None, st["expert_count"][0], 10, dw, dl, 3, False)
    part, _ = ref.gradient(0, True, 1.0, v, idx, None, st["expert_count"][0], 10, dw, None, 3, False)
    assert_within(full.float(), full, gb)
    for got, want, b in ((w * 1.001, w, bound), (part, full, gb), (full.roll(1, 0), full, gb)):
        with pytest.raises(AssertionError):
            assert_within(got, want, b)


def test_fp4_workspace_where_rows_stay_apart():
    """Many tiles: the workspace also holds an fp32 row for each entry; few: the hidden rows alone."""
    q = Q(C=256, N=128)
    for p, rows in ((P(T=63, E=64, K=3, H=256), True), (P(T=5, E=8, K=3, H=256), False)):
        entries = p.num_tokens * 3
        hidden = 256 + entries * q.out_features * 2
        need = ep.ep_moe_tokens_workspace_bytes(p, q)
        assert need == ((hidden + 255) // 256 * 256 + entries * 256 * 4 if rows else hidden)
        assert tokens_fp4(p=p, q=q, n=need - 1) == BAD


def test_reference_fp4_round_trip():
    g = torch.Generator().manual_seed(4)
    w = torch.randn(6, 96, generator=g)
    codes, sf = fp4.quantise(w)
    v = fp4.values(codes, sf)
    again = fp4.quantise(v)
    assert torch.equal(fp4.values(*again), v)
    top = w.abs().view(6, 3, 32).amax(-1, keepdim=True)
    assert ((v.view(6, 3, 32) - w.view(6, 3, 32)).abs() <= top / 4).all()
    assert fp4.values(torch.tensor([[0x1F] * 16], dtype=torch.uint8), torch.tensor([[128]], dtype=torch.uint8))[0, :2].tolist() == [-12.0, 1.0]
