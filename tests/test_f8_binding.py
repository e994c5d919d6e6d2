"""What the binding of the 8-bit calls refuses by shape before it looks at where
a tensor lies, so that these run without a GPU: a call that passed would go on
to refuse CPU tensors in other words."""
import pytest
import torch

F8 = torch.float8_e4m3fn
E, K, H, T = 8, 2, 64, 12


@pytest.fixture(scope="module")
def ep():
    from combine_ep_prepare_gb300 import build
    build.build()
    import combine_ep_prepare_gb300 as ep
    return ep


@pytest.fixture(scope="module")
def layer(ep):
    lid, size = ep.ep_register_layer(E, K, H, 16, 4)
    return ep.EpHandle(lid, torch.empty(size, dtype=torch.uint8)), ep.ep_recv_capacity(lid)


def dispatch_arguments(ep, rows, name=None, shape=None, width=H):
    a = dict(topk_idx=torch.zeros(T, K, dtype=torch.int64), tokens=torch.zeros(T, width, dtype=torch.uint8).view(F8),
             scales=torch.zeros(T, ep.scale_columns(width)), topk_weights=torch.zeros(T, K),
             recv_tokens=torch.zeros(rows, width, dtype=torch.uint8).view(F8),
             recv_scales=torch.zeros(rows, ep.scale_columns(width)), recv_topk_weights=torch.zeros(rows))
    if name is not None:
        a[name] = torch.zeros(*shape, dtype=a[name].dtype)
    return a


@pytest.mark.parametrize("name,shape", [("topk_idx", (T - 1, K)), ("topk_idx", (T, K + 1)), ("topk_idx", (T * K,)), ("topk_weights", (T, K - 1)),
                                        ("topk_weights", (T - 1, K)), ("recv_topk_weights", (T,))])
def test_dispatch_takes_the_layers_shapes_alone(ep, layer, name, shape):
    h, rows = layer
    with pytest.raises(ValueError, match="%s (must be )?\\[" % name):
        ep.ep_dispatch_f8(h, **dispatch_arguments(ep, rows, name, shape))


@pytest.mark.parametrize("width", [H - 16, H + 16])
def test_dispatch_takes_tokens_of_the_layers_width_alone(ep, layer, width):
    h, rows = layer
    with pytest.raises(ValueError, match="tokens must be \\[%d, %d\\]" % (T, H)):
        ep.ep_dispatch_f8(h, **dispatch_arguments(ep, rows, width=width))


def test_dispatch_of_the_layers_shapes_gets_as_far_as_the_device(ep, layer):
    h, rows = layer
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        ep.ep_dispatch_f8(h, **dispatch_arguments(ep, rows))
