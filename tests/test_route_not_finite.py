"""What one NaN or +inf logit does to its token's weights, statistics and gradient."""
import math

import pytest
import torch

import route_reference as ref
from product_reference import assert_within
from test_product import ep  # noqa: F401
from test_route import Call

pytestmark = pytest.mark.gpu
E, K, SCALE = 40, 4, 2.5


def rows(T, bf16=False):
    """T tokens of which 3 has a NaN and 5 a +inf."""
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(T))
    logits = logits.bfloat16().float() if bf16 else logits
    logits[3, 7], logits[5, 9] = math.nan, math.inf
    return logits.bfloat16() if bf16 else logits


@pytest.mark.parametrize("T,bf16", [(12, False), (12, True), (1100, False)])
@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("biased", [True, False])
def test_softmax_weights(ep, T, bf16, normalise, biased):  # noqa: F811
    logits = rows(T, bf16)
    c = Call(ep, logits, K, ref.SOFTMAX, normalise, SCALE, torch.linspace(-0.1, 0.1, E) if biased else None)
    idx, w = c.route()
    if biased:
        assert (idx[[3, 5]] == -1).all() and not w[[3, 5]].any()
    else:
        want = ref.choose(ref.SOFTMAX, logits, None, None, K)
        assert torch.equal(idx, want) and idx[5, 0] == 9 and 7 not in idx[3].tolist()
        assert torch.isnan(w[5]).all()
        if normalise:
            v = logits[3, idx[3].long()].double()
            assert ((w[3].double() - SCALE * torch.softmax(v, 0)).abs() <= SCALE * 64 * 2.0 ** -23).all()
        else:
            assert torch.isnan(w[3]).all()
    rest = [t for t in range(T) if t not in (3, 5)]
    assert torch.isfinite(w[rest]).all() and (idx[rest] >= 0).all()


@pytest.mark.parametrize("T,bf16", [(12, False), (12, True), (1100, False)])
@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("biased", [True, False])
def test_sigmoid_weights(ep, T, bf16, normalise, biased):  # noqa: F811
    logits, bias = rows(T, bf16), torch.linspace(-0.1, 0.1, E)
    idx, w = Call(ep, logits, K, ref.SIGMOID, normalise, SCALE, bias if biased else None).route()
    key = torch.sigmoid(logits[[3, 5]].double()) + bias.double() if biased else logits[[3, 5]].double()
    key[torch.isnan(key)] = -math.inf
    for row, k in zip((3, 5), key):
        assert idx[row].tolist() == torch.sort(k, descending=True, stable=True).indices[:K].tolist()
        s = torch.sigmoid(logits[row, idx[row].long()].double())
        want = SCALE * (s / s.sum() if normalise else s)
        assert ((w[row].double() - want).abs() <= want * 64 * 2.0 ** -23).all()
    if not biased:
        assert idx[5, 0] == 9


@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("row", [3, 5, None])
def test_statistics_and_gradient(ep, kind, row):  # noqa: F811
    logits = rows(1100)
    mask = torch.ones(1100, dtype=torch.uint8)
    for other in (3, 5):
        if other != row:
            mask[other] = 0
    c = Call(ep, logits, K, kind, mask=mask)
    idx, _ = c.route(stats=True)
    count, tokens, prob, losses = (t[:-1].cpu() for t in c.stats)
    assert int(tokens) == int(mask.sum())
    spoilt = row == 3 or (row == 5 and kind == ref.SOFTMAX)
    assert torch.isnan(prob).all() if spoilt else torch.isfinite(prob).all()
    assert bool(torch.isnan(losses[0])) == spoilt and bool(torch.isnan(losses[1])) == (row is not None)
    dw = torch.randn(1100, K, generator=torch.Generator().manual_seed(2))
    for dl in (None, torch.tensor([1.0, 0.1])):
        got = c.backward(idx, count, tokens, dw, dl)
        for t in (3, 5):
            assert torch.isnan(got[t]).all() if t == row else not got[t].any()
        rest = [t for t in range(1100) if t not in (3, 5)]
        plain = ref.gradient(kind, True, 1.0, logits[rest], idx[rest], None, count, tokens, dw[rest], dl, K, False)
        assert_within(got[rest], *plain)
