"""Host-side refusals of the experts' products, the few-token layer and the
combine's gradient: nothing is enqueued, so no GPU is needed.  And the 64-bit
forms that the GPU tests compare with, against plain torch."""
import ctypes

import pytest
import torch

import combine_ep_get_amd as ep
import product_reference as ref

A = 1 << 20  # an aligned address that is never dereferenced
BAD = ep.EP_ERR_INVALID_ARG


def P(**kw):
    base = dict(T=64, H=256, E=8, K=2, R=2, G=1, A=1, S=128)
    base.update(kw)
    return ep.Problem.make(**base)


def Q(C=256, N=128, act=ep.EP_ACT_SWIGLU, reserved=0):
    q = ep.Product.make(C, N, act)
    q.reserved = reserved
    return q


def call(name, p, q, *args):
    return getattr(ep.load(), name)(ctypes.byref(p), ctypes.byref(q), *args)


def product(p=None, q=None, x=A, count=A, offset=A, w=A, bias=A, res=A, pre=A, out=A):
    return call("ep_expert_product", p or P(), q or Q(), x, count, offset, w, bias, res, pre, out, None)


def product_fp8(p=None, q=None, x=A, sf=A, ts=2, hs=1, count=A, offset=A, w=A, wsf=A, bias=A, res=A, out=A):
    return call("ep_expert_product_fp8", p or P(), q or Q(), x, sf, ts, hs, count, offset, w, wsf, bias, res, out, None)


def backward(p=None, q=None, dout=A, pre=A, x=A, count=A, offset=A, w=A, dpre=A, dx=A, dw=A, acc=A, db=A, ws=A, n=1 << 30):
    return call("ep_expert_product_backward", p or P(), q or Q(), dout, pre, x, count, offset, w, dpre, dx, dw, acc, db,
                ws, n, None)


def tokens(p=None, q=None, x=A, idx=A, tw=A, w1=A, b1=A, w2=A, b2=A, res=A, out=A, ws=A, n=1 << 30):
    return call("ep_moe_tokens", p or P(), q or Q(), x, idx, tw, w1, b1, w2, b2, res, out, ws, n, None)


def tokens_fp8(p=None, q=None, x=A, idx=A, tw=A, w1=A, s1=A, b1=A, w2=A, s2=A, b2=A, res=A, out=A, ws=A, n=1 << 30):
    return call("ep_moe_tokens_fp8", p or P(), q or Q(), x, idx, tw, w1, s1, b1, w2, s2, b2, res, out, ws, n, None)


def combine(p=None, dout=A, y=A, slot=A, tw=A, dy=A, dw=A):
    return ep.load().ep_combine_backward(ctypes.byref(p or P()), dout, y, slot, tw, dy, dw, None)


ALL = (product, product_fp8, backward, tokens, tokens_fp8)


@pytest.mark.parametrize("fn", ALL, ids=lambda f: f.__name__)
def test_bad_problems_and_products(fn):
    for bad in (dict(E=9), dict(K=0), dict(H=250), dict(T=-1)):
        assert fn(p=P(**bad)) == BAD, bad
    for bad in (Q(C=0), Q(C=252), Q(N=4), Q(N=130), Q(C=(1 << 16) + 128), Q(N=(1 << 16) + 128), Q(act=-1), Q(act=6),
                Q(reserved=1)):
        assert fn(q=bad) == BAD, (bad.in_features, bad.out_features, bad.activation)
    # a weight of more than 2^31 values: 32768 outputs, both halves of a gate
    assert fn(q=Q(C=32768 + 128, N=32768), p=P(H=32768 + 128)) == BAD
    assert ep.load().ep_expert_product(ctypes.byref(P()), None, A, A, A, A, A, A, A, A, None) == BAD


@pytest.mark.parametrize("fn,names", [
    (product, "x w bias res pre out"), (product_fp8, "x w bias res out"),
    (backward, "dout pre x w dpre dx dw acc db ws"), (tokens, "x w1 b1 w2 b2 res out ws"),
    (tokens_fp8, "x w1 b1 w2 b2 res out ws")], ids=lambda v: getattr(v, "__name__", ""))
def test_misaligned_pointers(fn, names):
    for name in names.split():
        assert fn(**{name: A + 8}) == BAD, name


@pytest.mark.parametrize("fn,names", [
    (product, "x w out count offset"), (product_fp8, "x w out sf wsf count offset"), (backward, "dout pre x w dpre ws"),
    (tokens, "x idx w1 w2 out ws"), (tokens_fp8, "x idx w1 s1 w2 s2 out ws")], ids=lambda v: getattr(v, "__name__", ""))
def test_missing_pointers(fn, names):
    for name in names.split():
        assert fn(**{name: None}) == BAD, name


def test_scalar_arrays_are_aligned_to_their_elements():
    for fn, names in ((product, "count offset"), (product_fp8, "sf wsf count offset"), (tokens, "idx tw"),
                      (tokens_fp8, "idx tw s1 s2")):
        for name in names.split():
            assert fn(**{name: A + 2}) == BAD, (fn.__name__, name)


def test_fp8_sizes_and_strides():
    for q in (Q(C=264), Q(N=136)):
        assert product_fp8(q=q) == BAD
    assert tokens_fp8(q=Q(C=264), p=P(H=264)) == BAD
    assert product_fp8(ts=0) == BAD and product_fp8(hs=0) == BAD


def test_dense_product_is_one_expert():
    dense = dict(count=None, offset=None)
    assert product(**dense) == BAD                                    # 8 experts
    assert product(p=P(E=1, R=1, K=2), **dense) == BAD                # two entries a token
    assert product(p=P(E=1, R=1, K=1, S=63), **dense) == BAD          # fewer rows than tokens
    assert product(p=P(E=1, R=1, K=1), count=A, offset=None) == BAD   # one array of the two


def test_backward_combinations():
    none = Q(act=ep.EP_ACT_NONE)
    assert backward(q=none, pre=A, dpre=None) == BAD       # pre means nothing without an activation
    assert backward(q=none, pre=None, dpre=A) == BAD
    need = ep.ep_product_workspace_bytes(P(), Q())
    assert need > 0 and backward(n=need - 1) == BAD
    assert ep.ep_product_workspace_bytes(P(), Q(C=32768, N=32768)) > 0       # 2^31 values exactly
    assert ep.ep_product_workspace_bytes(P(), Q(C=32768, N=32768 + 8)) == 0
    assert ep.ep_product_workspace_bytes(P(), Q(C=4)) == 0 and ep.ep_product_workspace_bytes(P(S=0), Q()) == 0


def test_few_token_limits():
    assert tokens(p=P(T=ep.EP_MOE_TOKENS_MAX + 1)) == BAD
    assert tokens(p=P(H=128)) == BAD                       # in_features is not the hidden size
    need = ep.ep_moe_tokens_workspace_bytes(P(), Q())
    assert need >= 64 * 2 * 128 * 2 and tokens(n=need - 1) == BAD and tokens(ws=A + 128) == BAD
    assert ep.ep_moe_tokens_workspace_bytes(P(T=129), Q()) == 0
    assert ep.ep_moe_tokens_workspace_bytes(P(T=0, S=0), Q()) > 0


def test_combine_backward_refusals():
    assert combine(p=P(S=0)) == BAD and combine(p=P(H=7)) == BAD
    for name in ("dout", "slot"):
        assert combine(**{name: None}) == BAD
    assert combine(y=None) == BAD                          # the weights' gradients read y
    for name in ("dout", "y", "dy"):
        assert combine(**{name: A + 8}) == BAD
    assert combine(slot=A + 2) == BAD and combine(dw=A + 2) == BAD
    assert combine(dy=None, dw=None) == ep.EP_OK and combine(p=P(T=0)) == ep.EP_OK


def test_nothing_to_do_is_ok_without_a_device():
    assert product(p=P(T=0), x=None, w=None, out=None) == ep.EP_OK
    assert product_fp8(p=P(T=0)) == ep.EP_OK


def test_binding_checks():
    p, q = P(), Q()
    rows, M = 256, 256
    with pytest.raises(ValueError, match="x: .* elements, the call uses 65536"):
        ep.ep_expert_product(p, q, torch.zeros(rows * 256 - 1, dtype=torch.bfloat16), A, A, A, None, None, None, A, stream=0)
    with pytest.raises(ValueError, match="weight: dtype"):
        ep.ep_expert_product(p, q, A, A, A, torch.zeros(8, M, 256), None, None, None, A, stream=0)
    with pytest.raises(ValueError, match="bias: dtype"):
        ep.ep_expert_product(p, q, A, A, A, A, torch.zeros(8, M, dtype=torch.bfloat16), None, None, A, stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        ep.ep_expert_product(p, q, A, A, A, A, None, torch.zeros(128, rows, dtype=torch.bfloat16).t(), None, A, stream=0)
    with pytest.raises(ValueError, match="out: a cpu tensor"):
        ep.ep_expert_product(p, q, A, A, A, A, None, None, None, torch.zeros(rows, 128, dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError, match="x_sf: 5 elements"):
        ep.ep_expert_product_fp8(p, q, A, torch.zeros(5), 2, 1, A, A, A, A, None, None, A, stream=0)
    with pytest.raises(ValueError, match="dweight: .* the call uses 524288"):
        ep.ep_expert_product_backward(p, q, A, A, A, A, A, A, A, None, torch.zeros(9, dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError, match="w1_fp8|w1: dtype"):
        ep.ep_moe_tokens_fp8(p, q, A, A, A, torch.zeros(8, M, 256), A, None, A, A, None, None, A, A, 1 << 30, stream=0)
    with pytest.raises(ValueError, match="topk_idx: dtype"):
        ep.ep_moe_tokens(p, q, A, torch.zeros(64, 2, dtype=torch.int64), A, A, None, A, None, None, A, A, 1 << 30, stream=0)
    with pytest.raises(ValueError, match="dweights: 127 elements"):
        ep.ep_combine_backward(p, A, A, A, A, A, torch.zeros(127), stream=0)
    with pytest.raises(ep.EpError, match="invalid argument"):
        ep.ep_expert_product(p, Q(act=9), A, A, A, A, None, None, None, A, stream=0)


def test_reference_activations_match_torch():
    v = torch.linspace(-9, 9, 1001, dtype=torch.float64)
    zero = torch.zeros_like(v)
    assert torch.allclose(ref.activate("silu", v, zero)[0], torch.nn.functional.silu(v), atol=1e-14)
    assert torch.allclose(ref.activate("gelu", v, zero)[0], torch.nn.functional.gelu(v), atol=1e-14)
    assert torch.equal(ref.activate("relu", v, zero)[0], torch.relu(v))
    pair = torch.cat([v, v.flip(0)])
    assert torch.allclose(ref.activate("swiglu", pair, torch.zeros_like(pair))[0], torch.nn.functional.silu(v) * v.flip(0), atol=1e-13)


def test_reference_layout_by_hand():
    idx = torch.tensor([[0, 3], [3, -1], [1, 0]])
    of, slot, counts, offset = ref.layout(idx, 4, 2, 4, 2)
    assert counts == [2, 1, 0, 2] and offset == [0, 2, 0, 0]
    assert of == {0: [0, 1], 1: [2], 2: [], 3: [4, 5]}
    assert slot.tolist() == [[0, 4], [5, -1], [2, 1]]


def test_reference_sees_a_mistake():
    """A result off by three bf16 steps, a row in another's place or a missing bias is outside the bound."""
    g = torch.Generator().manual_seed(0)
    x, w, b = torch.randn(6, 64, generator=g).bfloat16(), torch.randn(16, 64, generator=g).bfloat16(), torch.randn(16, generator=g)
    o, bound, _, _ = ref.product("silu", x, w, b)
    ref.assert_within(o.bfloat16(), o, bound)
    for wrong in (o * (1 + 3 * 2.0 ** -7), o.roll(1, 0), ref.product("silu", x, w)[0]):
        with pytest.raises(AssertionError):
            ref.assert_within(wrong.bfloat16(), o, bound)
