"""An FP8 layer as a user strings it together: quantise, layout and dispatch of
e4m3 rows, up product, quantise the receive buffer's hidden rows, down
product, combine."""
import pytest
import torch

import product_reference as ref
from test_product import ep, marked, normal  # noqa: F401

pytestmark = pytest.mark.gpu


def values(codes, sf):
    return codes.cpu().view(torch.float8_e4m3fn).double() * sf.cpu().double().repeat_interleave(128, -1)


@pytest.mark.parametrize("T,H,I,E,K,R", [(9, 256, 128, 8, 2, 2), (100, 384, 256, 16, 4, 4), (600, 128, 384, 4, 2, 1)])
def test_fp8_layer(ep, T, H, I, E, K, R):  # noqa: F811
    g = torch.Generator().manual_seed(T)
    idx = torch.rand(T, E, generator=g).topk(K, 1).indices.int()
    idx[T // 2, 0] = -1
    tw, x = torch.softmax(torch.randn(T, K, generator=g), 1), normal(g, T, H)
    w1, w2 = ((torch.randn(*s, generator=g) * 64).to(torch.float8_e4m3fn) for s in ((E, 2 * I, H), (E, H, I)))
    s1 = (torch.rand(E, 2 * I // 128, H // 128, generator=g) + 0.5) * (H ** -0.5 / 64)
    s2 = (torch.rand(E, H // 128, I // 128, generator=g) + 0.5) * (I ** -0.5 / 64)
    d_idx, d_tw, d_x, d_w1, d_w2, d_s1, d_s2 = (t.cuda() for t in (idx, tw, x, w1, w2, s1, s2))
    p = ep.Problem.make(T, H, E, K, R, 1, 1, 1)
    p.rank_stride_rows = ep.ep_rank_stride_hint(p)
    rows, bufs = p.num_rows, ep.alloc_layout(p)
    seg, u8 = (bufs.expert_count, bufs.expert_offset), dict(dtype=torch.uint8, device="cuda")
    xq, xs = torch.empty(T, H, **u8), torch.empty(T, H // 128, device="cuda")
    recv, rsf = torch.zeros(rows, H, **u8), torch.zeros(rows, H // 128, device="cuda")
    hq, hs = torch.empty(rows, I, **u8), torch.empty(rows, I // 128, device="cuda")
    h, y, out = marked(rows, I), marked(rows, H), marked(T, H)
    ep.ep_quantize_fp8(p, d_x, xq, xs)
    ep.ep_layout_dispatch_fp8(p, d_idx, *bufs.args(), None, xq, xs, d_tw, recv, rsf, H // 128, 1)
    up, down = ep.Product.make(H, I, ep.EP_ACT_SWIGLU), ep.Product.make(I, H)
    ep.ep_expert_product_fp8(p, up, recv, rsf, H // 128, 1, *seg, d_w1, d_s1, None, None, h)
    # the hidden rows are the receive buffer's: a problem of R*S rows of I channels
    hidden = ep.Problem.make(rows, I, 1, 1, 1, 1, 1, rows)
    ep.ep_quantize_fp8(hidden, h, hq, hs)
    ep.ep_expert_product_fp8(p, down, hq, hs, I // 128, 1, *seg, d_w2, d_s2, None, None, y)
    ep.ep_combine(p, y, bufs.token_slot, d_tw, out)
    # Every step against the 64-bit form of what the step before left ...
    of, slot, _, _ = ref.layout(idx, E, R, p.rank_stride_rows)
    rv, hv, yv = values(recv, rsf), values(hq, hs), y.cpu()
    xv = values(xq, xs)
    for e, r in of.items():
        one = lambda w, s: w[e].double() * s[e].double().repeat_interleave(128, -1).repeat_interleave(128, -2)  # noqa: E731
        # the product of codes: what linear() adds for e4m3 blocks, on the same magnitudes
        v, verr = ref.linear(rv[r], one(w1, s1), None)
        verr = verr + (rv[r].abs() @ one(w1, s1).abs().t()) * ref.FP8_BLOCK
        o, oerr = ref.activate("swiglu", v, verr)
        ref.assert_within(h[r], o, ref.rounded(o, oerr), f"h of expert {e}")
        hb = h[r].cpu().double()
        # a code is off by half a step: 2^-4 of the value, or 2^-10 of the scale below the normal codes; fp32 scaling on top
        step = hs[r].cpu().double().repeat_interleave(128, -1) * 2.0 ** -10
        ref.assert_within(hv[r], hb, (2.0 ** -4 + 4 * ref.ULP32) * hb.abs() + step, f"codes of expert {e}")
        v, verr = ref.linear(hv[r], one(w2, s2), None)
        verr = verr + (hv[r].abs() @ one(w2, s2).abs().t()) * ref.FP8_BLOCK
        ref.assert_within(yv[r], v, ref.rounded(v, verr), f"y of expert {e}")
    ok = slot >= 0
    for t in range(T):
        at = slot[t][ok[t]].long()
        terms = tw[t][ok[t]].double()[:, None] * yv[at].double()
        v = terms.sum(0)
        ref.assert_within(out[t], v, ref.rounded(v, (K + 2) * ref.ULP32 * terms.abs().sum(0)), f"token {t}")
        # ... and the entries' rows are their tokens'
        assert torch.equal(rv[at], xv[t].expand(len(at), H))
