"""The combine's gradient on batches that need more than one launch, and on
the kernel that takes large batches."""
import pytest
import torch

import product_reference as ref
from test_product import Routed, ep, marked, normal, untouched  # noqa: F401

pytestmark = pytest.mark.gpu


def test_more_tokens_than_one_launch_holds(ep):  # noqa: F811
    """2^26 + 5 tokens: 64 threads each would be more than a launch can count in 32 bits."""
    T, H, rows = (1 << 26) + 5, 8, 16
    p = ep.Problem.make(T, H, 1, 1, 1, 1, 1, rows)
    dout = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    y = torch.arange(rows, device="cuda").bfloat16()[:, None].repeat(1, H)
    slot = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    w = torch.ones(T, 1, device="cuda")
    # first and last tokens, and those around 2^23 (a launch's tokens) and 2^26
    at = [0, 1, (1 << 23) - 2, (1 << 23) - 1, 1 << 23, (1 << 26) - 1, 1 << 26, T - 1]
    for i, t in enumerate(at):
        slot[t], w[t], dout[t] = i + 1, i + 2, i - 3
    dy, dw = torch.full((rows, H), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, 1), 7.0, device="cuda")
    ep.ep_combine_backward(p, dout, y, slot, w, dy, dw)
    # small whole numbers: exact in bf16 and fp32
    want = torch.zeros(T, 1, device="cuda")
    want_dy = torch.full((rows, H), 9.0)
    for i, t in enumerate(at):
        want[t] = (i - 3) * (i + 1) * H
        want_dy[i + 1] = (i - 3) * (i + 2)
    assert torch.equal(dw, want)
    assert torch.equal(dy.float().cpu(), want_dy)


@pytest.mark.parametrize("K", [3, 9])
@pytest.mark.parametrize("weights", [True, False])
def test_entries_about_the_end_of_a_launch(ep, K, weights):  # noqa: F811
    """2^23 + 40 tokens, those around 2^23 with slots: each token's entries, weights and results stay its own."""
    T, H, n = (1 << 23) + 40, 8, 64
    first = (1 << 23) - 24
    g = torch.Generator().manual_seed(K)
    rows = n * K
    slot = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    slot[first:] = torch.randperm(rows, generator=g).int().view(n, K).cuda()
    dout, w = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, K, device="cuda")
    d, y, wt = normal(g, n, H), normal(g, rows, H), torch.rand(n, K, generator=g)
    dout[first:], w[first:] = d.cuda(), wt.cuda()
    dy, dw = marked(rows, H), torch.full((T, K), 7.0, device="cuda")
    p = ep.Problem.make(T, H, 16, K, 1, 1, 1, rows)
    ep.ep_combine_backward(p, dout, y.cuda(), slot, w if weights else None, dy, dw)
    some = slot[first:].cpu()
    ok, vy, by, vw, bw = ref.combine_backward(d, y, some, wt if weights else None, rows)
    ref.assert_within(dy[some[ok].long().cuda()], vy[ok], by[ok], "dy")
    ref.assert_within(dw[first:], vw, bw, "dweights")
    assert not dw[:first].any()


@pytest.mark.parametrize("T,H,E,K,R,empty", [
    (4200, 264, 32, 8, 4, 0.1),    # eight entries at a time
    (4300, 136, 24, 5, 2, 0.3),    # a group that is not full
    (4100, 136, 40, 20, 4, 0.1),   # three groups, the last of four
    (4096, 1032, 16, 12, 1, 0.0),  # the smallest batch of this kernel, more than one wave
    (5000, 72, 8, 3, 2, 0.5),      # four at a time
    (4095, 136, 16, 12, 2, 0.1),   # the largest of one entry a workgroup
])
def test_large_batches(ep, T, H, E, K, R, empty):  # noqa: F811
    r = Routed(ep, T, E, K, R, hidden=H, empty=empty, seed=T + K)
    g = torch.Generator().manual_seed(K)
    dout, y, w = normal(g, T, H), normal(g, r.rows, H), torch.randn(T, K, generator=g)
    # rows that no slot names are not read: row 0 may be one of them
    unused = torch.ones(r.rows, dtype=torch.bool)
    unused[r.used] = False
    y[unused] = float("nan")
    dy, dw = marked(r.rows, H), torch.full((T, K), 7.0, device="cuda")
    cd, cy, cw = dout.cuda(), y.cuda(), w.cuda()
    ep.ep_combine_backward(r.p, cd, cy, r.bufs.token_slot, cw, dy, dw)
    ok, vy, by, vw, bw = ref.combine_backward(dout, y.nan_to_num(0.0), r.slot, w, r.rows)
    at = r.slot[ok].long().cuda()
    ref.assert_within(dy[at], vy[ok], by[ok], "dy")
    ref.assert_within(dw, vw, bw, "dweights")
    assert untouched(dy, at)
    # each alone, and dy in y's place: the same bits
    dy2, dw2 = marked(r.rows, H), torch.empty_like(dw)
    ep.ep_combine_backward(r.p, cd, None, r.bufs.token_slot, cw, dy2, None)
    assert torch.equal(dy2.view(torch.int16), dy.view(torch.int16))
    ep.ep_combine_backward(r.p, cd, cy, r.bufs.token_slot, cw, None, dw2)
    assert torch.equal(dw2, dw)
    for _ in range(3):
        cy, dw2 = y.cuda(), torch.empty_like(dw)
        ep.ep_combine_backward(r.p, cd, cy, r.bufs.token_slot, cw, cy, dw2)
        assert torch.equal(cy.view(torch.int16)[at], dy.view(torch.int16)[at]) and torch.equal(dw2, dw)
        assert torch.isnan(cy[unused.cuda()]).all()


@pytest.mark.parametrize("T", [40, 4100])
def test_first_row_belongs_to_another_token(ep, T):  # noqa: F811
    """Row 0 is named by the last token, in whose place its gradient is
    written, while every other token has empty entries."""
    H, K = 136, 6
    g = torch.Generator().manual_seed(T)
    slot = torch.full((T, K), -1, dtype=torch.int32)
    slot[:, 2] = torch.arange(T, 0, -1) - 1
    p = ep.Problem.make(T, H, 8, K, 1, 1, 1, T)
    dout, y = normal(g, T, H), normal(g, T, H)
    cy, dw = y.cuda(), torch.full((T, K), 7.0, device="cuda")
    ep.ep_combine_backward(p, dout.cuda(), cy, slot.cuda(), None, cy, dw)
    ok, vy, by, vw, bw = ref.combine_backward(dout, y, slot, None, T)
    assert torch.equal(cy.cpu(), dout.flip(0))
    ref.assert_within(dw, vw, bw, "dweights")
