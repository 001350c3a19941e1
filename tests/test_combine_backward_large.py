"""The combine's gradient on batches that need more than one launch, and on
the kernel that takes large batches."""
import pytest
import torch

from test_product import ep  # noqa: F401

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
