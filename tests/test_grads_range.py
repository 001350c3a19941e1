"""The gradients' clipping at the ends of fp32's range.

Bounds: as for other gradients (the factor's and the product's half steps of fp32, bf16's own of 2^-8, and half a step
below the normal numbers), however small the factor is."""
import math

import pytest
import torch

from test_grads import BF, clip
from test_product import ep  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size,max_norm", [(1e38, 1e-6), (3e38, 1e-30), (3e38, 1.0), (1e30, 2e-8), (1e25, 1e-38), (3e38, 1e-45)])
@pytest.mark.parametrize("shift", [0, 1])
def test_factors_below_the_normal_numbers(ep, size, max_norm, shift):  # noqa: F811
    """max_norm / norm is below 2^-126 or about it, and the products are not all 0."""
    g = torch.Generator().manual_seed(int(math.log10(size)))
    n = 20011
    wide = (torch.rand(n, generator=g) * 2 - 1) * size
    grads = [wide.cuda(), wide[:999].to(BF).cuda(), (wide * 1e-20).cuda()]
    outs = [torch.full((n + 8,), 77.0, dtype=t.dtype, device="cuda")[shift:shift + t.numel()] for t in grads]
    held = [t.clone() for t in grads]
    norm, square = clip(ep, grads, outs, max_norm)
    factor = torch.tensor(max_norm).double().item() / math.sqrt(square)
    assert 0 < factor < 2.0 ** -122
    for o, b in zip(outs, grads):
        want = b.double() * factor
        tol = want.abs() * (2.0 ** -23 + (2.0 ** -8 if o.dtype == BF else 0)) + (2.0 ** -133 if o.dtype == BF else 2.0 ** -149)
        assert ((o.double() - want).abs() <= tol).all()
    assert all(torch.equal(a, b) for a, b in zip(grads, held))
    # in place: the same bits
    clip(ep, grads, grads, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))


def test_norms_past_fp32(ep):  # noqa: F811
    """A norm of 2^128 and more is finite in 64 bits and scales; only its fp32 output is infinite."""
    grads = [torch.full((5000,), 2.0 ** 127, device="cuda"), torch.full((33,), -2.0 ** 127, device="cuda", dtype=BF)]
    outs = [torch.empty_like(t) for t in grads]
    norm, square = clip(ep, grads, outs, 4.0)
    assert math.isinf(norm) and square == 5033 * 2.0 ** 254
    want = 4.0 / math.sqrt(5033)
    assert ((outs[0].double() - want).abs() <= want * 2.0 ** -23).all()
    assert ((outs[1].double() + want).abs() <= want * (2.0 ** -23 + 2.0 ** -8)).all()
