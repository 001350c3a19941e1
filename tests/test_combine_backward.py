"""The combine's gradient on the GPU against its 64-bit form."""
import pytest
import torch

import product_reference as ref
from test_product import Routed, ep, marked, normal, untouched  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,E,K,R", [(1, 8, 1, 1, 1), (5, 72, 8, 3, 2), (64, 7168, 32, 8, 4), (700, 264, 16, 4, 4),
                                       (3000, 520, 8, 2, 1), (33, 40000, 4, 2, 1), (9, 136, 64, 32, 8)])
@pytest.mark.parametrize("weights", [True, False])
def test_combine_backward(ep, T, H, E, K, R, weights):  # noqa: F811
    r = Routed(ep, T, E, K, R, hidden=H, empty=0.1 if T > 4 else 0.0, seed=T, S=None if T < 1000 else 4000)
    g = torch.Generator().manual_seed(T)
    dout, y = normal(g, T, H), normal(g, r.rows, H)
    w = torch.randn(T, K, generator=g) if weights else None
    cw = w.cuda() if weights else None
    dy, dw = marked(r.rows, H), torch.full((T, K), 7.0, device="cuda")
    cd, cy = dout.cuda(), y.cuda()
    ep.ep_combine_backward(r.p, cd, cy, r.bufs.token_slot, cw, dy, dw)
    ok, vy, by, vw, bw = ref.combine_backward(dout, y, r.slot, w, r.rows)
    at = r.slot[ok].long()
    ref.assert_within(dy[at.cuda()], vy[ok], by[ok], "dy")
    ref.assert_within(dw, vw, bw, "dweights")
    assert untouched(dy, at.cuda())
    # one at a time, and dy in y's place: the same bits
    dy2, dw2 = marked(r.rows, H), torch.empty_like(dw)
    ep.ep_combine_backward(r.p, cd, None, r.bufs.token_slot, cw, dy2, None)
    ep.ep_combine_backward(r.p, cd, cy, r.bufs.token_slot, cw, None, dw2)
    assert torch.equal(dy2.view(torch.int16), dy.view(torch.int16)) and torch.equal(dw2, dw)
    ep.ep_combine_backward(r.p, cd, cy, r.bufs.token_slot, cw, cy, dw2)
    assert torch.equal(cy[at.cuda()], dy[at.cuda()]) and torch.equal(dw2, dw)


def test_slots_outside_the_buffer_are_skipped(ep):  # noqa: F811
    p = ep.Problem.make(3, 16, 4, 2, 1, 1, 1, 5)
    slot = torch.tensor([[0, -1], [5, 2 ** 31 - 1], [4, -2 ** 31]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(0)
    dout, y = normal(g, 3, 16).cuda(), normal(g, 5, 16).cuda()
    dy, dw = marked(5, 16), torch.full((3, 2), 7.0, device="cuda")
    ep.ep_combine_backward(p, dout, y, slot, None, dy, dw)
    assert untouched(dy, [0, 4]) and torch.equal(dy[[0, 4]], dout[[0, 2]])
    assert (dw == 0).cpu().tolist() == [[False, True], [True, True], [False, True]]


def test_infinities_stay_in_their_row(ep):  # noqa: F811
    r = Routed(ep, 6, 4, 2, hidden=64, S=20)
    g = torch.Generator().manual_seed(0)
    dout, y = normal(g, 6, 64).cuda(), normal(g, r.rows, 64).cuda()
    dy, dw = marked(r.rows, 64), torch.empty(6, 2, device="cuda")
    unused = [i for i in range(r.rows) if i not in r.used]
    y[unused] = float("nan")
    dout[3, 5] = float("inf")
    ep.ep_combine_backward(r.p, dout, y, r.bufs.token_slot, None, dy, dw)
    assert torch.isfinite(dw[[0, 1, 2, 4, 5]]).all() and not torch.isfinite(dw[3]).any()
    assert untouched(dy, r.used)
