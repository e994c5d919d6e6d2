"""What a MoELayer's backward may follow: a forward that ended, and nothing else."""
import pytest
import torch

from tests.test_moe_layer_gpu import moe, problem  # noqa: F401

pytestmark = pytest.mark.gpu


def test_backward_after_a_refused_decode_is_refused(moe):  # noqa: F811
    """An fp32 layer has no 4-bit products: decode raises after it has routed
    another batch into the layer's buffers."""
    E, K, H, F, T = 4, 2, 64, 64, 10
    x, gate, w13, w2, grad = problem(E, K, H, F, T, torch.float32)
    layer = moe.MoELayer(E, K, H, F, T, dtype=torch.float32)
    layer.forward(x, gate, w13, w2)
    with pytest.raises(Exception, match="bf16 and fp16"):
        layer.decode(x.flip(0).contiguous(), gate, layer.quantize(w13, w2, 32))
    with pytest.raises(ValueError, match="last forward"):
        layer.backward(grad, w13, w2, gate)


@pytest.mark.parametrize("fault", ["weights of another layer", "a bias", "tokens of another type"])
def test_backward_after_a_refused_forward_is_refused(moe, fault):  # noqa: F811
    E, K, H, F, T = 4, 2, 64, 64, 10
    x, gate, w13, w2, grad = problem(E, K, H, F, T, torch.bfloat16)
    layer = moe.MoELayer(E, K, H, F, T)
    first = layer.forward(x, gate, w13, w2)
    with pytest.raises(Exception):
        if fault == "a bias":  # softmax takes none
            layer.forward(x, gate, w13, w2, bias=torch.zeros(E, device="cuda"))
        elif fault == "tokens of another type":
            layer.forward(x.float(), gate, w13, w2)
        else:
            layer.forward(x, gate, w13, w2[:, :, :32].contiguous())
    with pytest.raises(ValueError, match="last forward"):
        layer.backward(grad, w13, w2, gate)
    # the layer goes on with the next forward
    assert torch.equal(layer.forward(x, gate, w13, w2), first)
    layer.backward(grad, w13, w2, gate)
