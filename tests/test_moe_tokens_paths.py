"""The few-token layer on the kernels that its large calls take: waves of the up
product that work alone (from 1024 pairs of an expert and 16 outputs), 16 and 32
columns at a time, and 32 outputs a workgroup of the down product (more than
64 tokens and 4096 channels)."""
import pytest
import torch

import product_reference as ref
from test_moe_tokens import problem
from test_product import ep, marked, normal  # noqa: F401

pytestmark = pytest.mark.gpu


def spread(E, T, K, seed):
    """ids [T,K], each expert once a token at most: experts 0 to 5 have 1, 16,
    17, 32, 33 and 64 entries, the others share what is left, one at least."""
    g = torch.Generator().manual_seed(seed)
    first = [n for n in (1, 16, 17, 32, 33, 64) if n <= T]
    idx = torch.full((T, K), -1, dtype=torch.int32)
    used = [0] * T
    for e, n in enumerate(first):
        # the tokens with most room
        for t in sorted(range(T), key=lambda t: (used[t], float(torch.rand(1, generator=g))))[:n]:
            idx[t, used[t]] = e
            used[t] += 1
    e = len(first)
    for t in range(T):
        while used[t] < K:
            if e >= E:
                e = len(first)
            if (idx[t] == e).any():
                break
            idx[t, used[t]] = e
            used[t] += 1
            e += 1
    counts = torch.bincount(idx[idx >= 0].long(), minlength=E)
    assert counts[:len(first)].tolist() == first and (counts > 0).all()
    return idx


CASES = [
    # T, H, I, E, K, act, bias, residual: up products with waves alone
    (128, 136, 264, 64, 8, "swiglu", True, True),
    (100, 264, 264, 64, 8, "geglu", False, False),
    (128, 200, 264, 64, 6, "silu", True, False),
    (128, 136, 272, 64, 4, "none", False, True),
    # 32 outputs a workgroup, the last one a quarter full (4104) or whole
    (65, 4104, 40, 8, 4, "swiglu", True, True),
    (128, 4104, 136, 8, 3, "gelu", True, False),
    (128, 4128, 72, 4, 2, "relu", False, True),
    # the widest with 16
    (128, 4096, 72, 4, 2, "silu", True, True),
    # both
    (128, 4104, 272, 64, 8, "swiglu", True, True),
]


def ids(T, E, K):
    g = torch.Generator().manual_seed(T)
    if E == 64:
        return spread(E, T, K, T)
    idx = torch.rand(T, E, generator=g).topk(K, 1).indices.int()
    idx[torch.rand(T, K, generator=g) < 0.1] = -1
    return idx


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])))
def test_tokens(ep, case):  # noqa: F811
    T, H, I, E, K, act, bias, residual = case
    idx = ids(T, E, K)
    p, q = problem(ep, T, H, E, K), ep.Product.make(H, I, ref.ACTS.index(act))
    assert E < 64 or E * ((I + 15) // 16) >= 1024
    M, g = q.weight_rows, torch.Generator().manual_seed(H)
    x, w1, w2 = normal(g, T, H), normal(g, E, M, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    b1, b2 = (torch.randn(E, M, generator=g), torch.randn(E, H, generator=g)) if bias else (None, None)
    res, tw = normal(g, T, H) if residual else None, torch.rand(T, K, generator=g)
    ws = torch.empty(ep.ep_moe_tokens_workspace_bytes(p, q), dtype=torch.uint8, device="cuda")
    d = [None if t is None else t.cuda() for t in (x, idx, tw, w1, b1, w2, b2, res)]
    out = marked(T, H)
    ep.ep_moe_tokens(p, q, *d, out, ws)
    assert ep.ep_read_status(ws) == ep.EP_OK
    want, bound = ref.tokens(act, x, idx, tw, w1, b1, w2, b2, res)
    ref.assert_within(out, want, bound)
    for _ in range(2):  # the same bits, into x itself
        again = d[0].clone()
        ep.ep_moe_tokens(p, q, again, *d[1:], again, ws)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16))


FP8_CASES = [
    (128, 256, 256, 64, 8, "swiglu", True),
    (100, 128, 384, 64, 6, "silu", False),
    (128, 4096, 128, 4, 2, "geglu", True),
    (65, 4224, 128, 8, 4, "none", True),
    (128, 4352, 128, 4, 2, "geglu", True),
    (128, 4224, 256, 64, 4, "swiglu", False),
]


@pytest.mark.parametrize("case", FP8_CASES, ids=lambda c: "-".join(map(str, c[:6])))
def test_tokens_fp8(ep, case):  # noqa: F811
    T, H, I, E, K, act, extras = case
    idx = ids(T, E, K)
    p, q = problem(ep, T, H, E, K), ep.Product.make(H, I, ref.ACTS.index(act))
    assert E < 64 or E * (I // 16) >= 1024
    M, g = q.weight_rows, torch.Generator().manual_seed(H)
    x = normal(g, T, H)
    w1, w2 = ((torch.randn(*s, generator=g) * 64).to(torch.float8_e4m3fn) for s in ((E, M, H), (E, H, I)))
    s1 = (torch.rand(E, M // 128, H // 128, generator=g) + 0.5) * (H ** -0.5 / 64)
    s2 = (torch.rand(E, H // 128, I // 128, generator=g) + 0.5) * (I ** -0.5 / 64)
    b1, b2 = (torch.randn(E, M, generator=g), torch.randn(E, H, generator=g)) if extras else (None, None)
    res, tw = normal(g, T, H) if extras else None, torch.rand(T, K, generator=g)
    ws = torch.empty(ep.ep_moe_tokens_workspace_bytes(p, q), dtype=torch.uint8, device="cuda")
    d = [None if t is None else t.cuda() for t in (x, idx, tw, w1, s1, b1, w2, s2, b2, res)]
    out = marked(T, H)
    ep.ep_moe_tokens_fp8(p, q, *d, out, ws)
    want, bound = ref.tokens(act, x, idx, tw, w1.float(), b1, w2.float(), b2, res, s1, s2)
    ref.assert_within(out, want, bound)
    again = d[0].clone()
    ep.ep_moe_tokens_fp8(p, q, again, *d[1:], again, ws)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
