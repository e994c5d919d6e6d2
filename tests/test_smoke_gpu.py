"""The smoke step's check of the MoE layer: it passes, and it sees a gradient
that is not the layer's.  The mistake is planted in the torch side."""
import pytest
import torch

import __graft_entry__ as entry
from combine_ep_prepare_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


def test_moe_layer_step_passes():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    entry._smoke_moe_layer(wl, torch)


@pytest.mark.parametrize("which,name", list(enumerate(["x", "gate", "w13", "w2"])))
@pytest.mark.parametrize("mistake", ["zeros", "sign"])
def test_moe_layer_step_sees_a_wrong_gradient(monkeypatch, which, name, mistake):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    right = torch.autograd.grad

    def wrong(*args, **kw):
        grads = list(right(*args, **kw))
        grads[which] = torch.zeros_like(grads[which]) if mistake == "zeros" else -grads[which]
        return tuple(grads)

    monkeypatch.setattr(torch.autograd, "grad", wrong)
    with pytest.raises(AssertionError, match="gradient of %s" % name):
        entry._smoke_moe_layer(wl, torch)
