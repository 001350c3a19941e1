"""MXFP4 weights at the top of the scales: exact while bf16 holds them, infinite from 2^128 on, NaN at byte 255."""
import pytest
import torch

import fp4_reference as fp4
from test_product import ep, marked  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,C", [(1, 32), (40, 288)])
@pytest.mark.parametrize("sf", [250, 251, 252, 253, 254, 255])
def test_top_scales(ep, rows, C, sf):  # noqa: F811
    """A weight row holds one code that is not 0 (each code, in every place of a scale's 32), and a token 1 in all its
    columns: the product is that value, and the 0 of the others adds nothing."""
    N = 512
    code, at = torch.arange(N) % 16, (torch.arange(N) // 16 * 37) % C
    codes = torch.zeros(N, C // 2, dtype=torch.uint8)
    codes[torch.arange(N), at // 2] = (code << 4 * (at % 2)).to(torch.uint8)
    scales = torch.full((N, C // 32), 127, dtype=torch.uint8)
    scales[torch.arange(N), at // 32] = sf
    want = fp4.values(codes, scales).sum(1)
    if sf < 255:
        want[want.abs() >= 2.0 ** 128] *= float("inf")
        assert int(torch.isinf(want).sum()) == {253: 4, 254: 8}.get(sf, 0) * N // 16
    p, q = ep.Problem.make(rows, 64, 1, 1, 1, 1, 1, rows), ep.Product.make(C, N)
    out = marked(rows, N)
    ep.ep_expert_product_fp4(p, q, torch.ones(rows, C).bfloat16().cuda(), None, None, codes.cuda(), scales.cuda(), None, None, out)
    got = out.cpu().double()
    if sf == 255:
        assert torch.isnan(got).all()
    else:
        assert torch.equal(got, want.expand(rows, N))
