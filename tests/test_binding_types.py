"""Element types of the arguments where torch lacks the newest ones."""
import pytest
import torch

from combine_ep_get_amd import _binding


@pytest.fixture
def fresh(monkeypatch):
    """The table of types as a process makes it on its first call."""
    monkeypatch.setattr(_binding, "_DTYPES", {})
    return monkeypatch


def test_types_that_torch_lacks_are_left_out(fresh):
    for name in ("float4_e2m1fn_x2", "float8_e8m0fnu"):
        if hasattr(torch, name):
            fresh.delattr(torch, name)
    with pytest.raises(ValueError, match="a cpu tensor"):  # the last check: the type was found
        _binding._arg(torch.zeros(4, dtype=torch.int32), "topk_idx", "int32", 4)
    for ctype in ("e2m1", "e8m0"):
        with pytest.raises(ValueError, match="a cpu tensor"):
            _binding._arg(torch.zeros(4, dtype=torch.uint8), "w", ctype, 4)
        with pytest.raises(ValueError, match="dtype torch.float32"):
            _binding._arg(torch.zeros(4), "w", ctype, 4)


def test_types_that_torch_has_are_taken(fresh):
    for name, ctype in (("float4_e2m1fn_x2", "e2m1"), ("float8_e8m0fnu", "e8m0")):
        if hasattr(torch, name):
            assert getattr(torch, name) in _binding._dtypes()[ctype]
