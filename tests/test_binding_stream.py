"""The stream that a call takes when none is given, with and without torch's private accessor."""
import types

import torch

from combine_ep_get_amd import _binding


def test_current_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=1234))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 70 + device, raising=False)
    assert _binding._stream(None) == 73
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert _binding._stream(None) == 1234


def test_given_stream():
    assert _binding._stream(0) == 0 and _binding._stream(types.SimpleNamespace(cuda_stream=5)) == 5
