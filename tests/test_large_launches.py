"""Batches whose launch would need 2^32 threads or more: refused, where the
grid would wrap and leave the last tokens without a workgroup."""
import pytest
import torch

from test_product import ep  # noqa: F401

pytestmark = pytest.mark.gpu


def test_too_many_threads_for_a_launch(ep):  # noqa: F811
    T, H, rows = 1 << 26, 512, 16
    wide = torch.empty(T * H, dtype=torch.bfloat16, device="cuda")  # 64 GiB, of which nothing is read or written
    slot = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    few = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
    p = ep.Problem.make(T, H, 1, 1, 1, 1, 1, rows)
    with pytest.raises(ep.EpError, match="ep_combine"):
        ep.ep_combine(p, few, slot, None, wide.view(T, H))
    with pytest.raises(ep.EpError, match="ep_dispatch"):
        ep.ep_dispatch(p, wide.view(T, H), None, slot, few, None, None)
    # narrow rows, several to a workgroup: 2^26 x 8 entries of 8 vectors
    p = ep.Problem.make(1 << 26, 64, 16, 8, 1, 1, 1, rows)
    slot = torch.full((1 << 26, 8), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(ep.EpError, match="ep_dispatch"):
        ep.ep_dispatch(p, wide[: (1 << 26) * 64].view(1 << 26, 64), None, slot, few, None, None)
    torch.cuda.synchronize()
    assert not few.any()
    del wide, slot
    torch.cuda.empty_cache()
