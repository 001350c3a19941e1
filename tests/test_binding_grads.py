"""Lists of gradients that the clipping has no defined result for."""
import pytest
import torch

import combine_ep_get_amd as ep


def test_the_same_gradient_twice():
    a, b = torch.zeros(4), torch.zeros(4)
    with pytest.raises(ValueError, match="tensors 0 and 2 are the same memory"):
        ep.Grads.make([a, b, a])
    with pytest.raises(ValueError, match="tensors 0 and 1 are the same memory"):
        ep.Grads.make([a, b], [a, a])
    with pytest.raises(ValueError, match="tensors 0 and 1 are the same memory"):
        ep.Grads.make([a, a.view(2, 2)])
    for ok in ([torch.zeros(0)] * 2, [a, a[1:]]):  # no values;  other addresses are the caller's to keep apart
        with pytest.raises(ValueError, match="a cpu tensor"):
            ep.Grads.make(ok)


@pytest.mark.gpu
def test_the_same_gradient_into_two_places():
    a = torch.randn(100, device="cuda")
    outs = [torch.empty_like(a) for _ in range(2)]
    one = ep.Grads.make([a, a], outs)
    square = torch.empty(1, dtype=torch.float64, device="cuda")
    ws = torch.empty(ep.ep_grad_workspace_bytes(one), dtype=torch.uint8, device="cuda")
    ep.ep_grad_square_sum(one, square, ws)
    ep.ep_grad_clip(one, square, 1.0)
    exact = 2 * float((a.double() ** 2).sum())
    assert abs(float(square) - exact) <= 2.0 ** -40 * exact
    assert torch.equal(*outs) and ((outs[0].double() - a.double() * exact ** -0.5).abs() <= a.abs() * 2.0 ** -23).all()
