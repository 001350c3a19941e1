"""The newer calls refuse a tensor of another device than the current one, whichever argument it is."""
import inspect

import pytest
import torch

import combine_ep_get_amd as ep
from test_product_abi import A, P, Q
from test_route_abi import R

CALLS = {
    "ep_expert_product_fp4": (P(), Q()), "ep_moe_tokens_fp4": (P(), Q()), "ep_route": (P(), R()),
    "ep_balance_loss": (P(), R()), "ep_route_backward": (P(), R()),
}
ARRAYS = [(name, a) for name in CALLS for a in list(inspect.signature(getattr(ep, name)).parameters)[2:]
          if a not in ("workspace_bytes", "stream", "bind")]


class Elsewhere:
    """A tensor of device 0, of which the binding gets no further than asking for its device."""

    def get_device(self):
        return 0


@pytest.mark.parametrize("name,array", ARRAYS)
def test_every_array(monkeypatch, name, array):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    fn = getattr(ep, name)
    args = {a: A for a in inspect.signature(fn).parameters if (name, a) in ARRAYS}
    args[array] = Elsewhere()
    if "workspace_bytes" in inspect.signature(fn).parameters:
        args["workspace_bytes"] = 1 << 30
    with pytest.raises(ValueError, match="device 0 with device 1 current"):
        fn(*CALLS[name], **args)


def test_the_gradients(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    none = ep.Grads.make([])
    for fn, args in ((ep.ep_grad_square_sum, (Elsewhere(), A, 1 << 30)), (ep.ep_grad_square_sum, (A, Elsewhere(), 1 << 30)),
                     (ep.ep_grad_clip, (Elsewhere(), 1.0)), (ep.ep_grad_clip, (A, 1.0, Elsewhere()))):
        with pytest.raises(ValueError, match="device 0 with device 1 current"):
            fn(none, *args)
    with pytest.raises(ValueError, match="device 0 with device 1 current"):
        ep.ep_grad_clip(ep.Grads((ep.Grad * 1)(), ([Elsewhere()], [Elsewhere()])), A, 1.0)


def test_host_tensors_are_named():
    """Also where no device is there to compare with."""
    with pytest.raises(ValueError, match="logits: a cpu tensor"):
        ep.ep_route(P(), R(), torch.zeros(64, 8), None, None, A, A, stream=None)
    with pytest.raises(ValueError, match="w_sf: a cpu tensor"):
        ep.ep_expert_product_fp4(P(), Q(), A, A, A, A, torch.zeros(1 << 20, dtype=torch.uint8), None, None, A)
