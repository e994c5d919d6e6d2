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


def f8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8).view(F8)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def products(ep, layer, rows, scales, w, w_scales, call):
    h, R = layer
    if call == "ep_expert_gemm_f8":
        ep.ep_expert_gemm_f8(h, rows, scales, w, w_scales, bf16(R, w.shape[1]))
    elif call == "ep_expert_gemm_f8_swiglu":
        ep.ep_expert_gemm_f8_swiglu(h, rows, scales, w, w_scales, act=bf16(R, w.shape[1] // 2))
    elif call == "ep_expert_dgrad_f8":
        ep.ep_expert_dgrad_f8(h, rows, scales, w, w_scales, bf16(R, w.shape[2]))
    else:
        ep.ep_expert_dgrad_f8_swiglu(h, rows, scales, w, w_scales, bf16(R, 2 * w.shape[2]), bf16(R, 2 * w.shape[2]))


CALLS = ["ep_expert_gemm_f8", "ep_expert_gemm_f8_swiglu", "ep_expert_dgrad_f8", "ep_expert_dgrad_f8_swiglu"]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("off", [(1, 0, 0), (0, 1, 0), (0, -1, 0), (0, 0, 1), (0, 0, -1)])
def test_products_take_weight_scales_of_their_blocks_alone(ep, layer, call, off):
    n, k = 256, 384
    rows = k if "gemm" in call else n
    x, xs = f8(layer[1], rows), torch.zeros(layer[1], ep.scale_columns(rows))
    shape = [E + off[0], n // 128 + off[1], k // 128 + off[2]]
    with pytest.raises(ValueError, match="w_scales must be \\[%d, %d, %d\\]" % (E, n // 128, k // 128)):
        products(ep, layer, x, xs, f8(E, n, k), torch.zeros(*shape), call)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        products(ep, layer, x, xs, f8(E, n, k), torch.zeros(E, n // 128, k // 128), call)


@pytest.mark.parametrize("columns,missing", [(4, 1), (3, 0), (8, 0)])
def test_receive_rows_have_scales_of_their_layers_capacity(ep, layer, columns, missing):
    h, R = layer
    with pytest.raises(ValueError, match="q_scales must be \\[>= %d rows, 4\\]" % R):
        ep.ep_expert_quantize(h, bf16(R, 256), f8(R, 256), torch.zeros(R - missing, columns))


@pytest.mark.parametrize("shape", [(3, 2), (3, 8), (2, 4)])
def test_rows_have_scales_of_their_blocks(ep, shape):
    with pytest.raises(ValueError, match="scales must be \\[3, 4\\]"):
        ep.ep_quantize_rows(torch.zeros(3, 256), f8(3, 256), torch.zeros(*shape))
    with pytest.raises(ValueError, match="scales must be \\[3, 4\\]"):
        ep.ep_rmsnorm(torch.zeros(3, 256), torch.zeros(256), q=f8(3, 256), scales=torch.zeros(*shape))
    with pytest.raises(ValueError, match="q must be \\[3, 256\\]"):
        ep.ep_quantize_rows(torch.zeros(3, 256), f8(3, 128), torch.zeros(3, 4))


@pytest.mark.parametrize("name,shape", [("weight", (128,)), ("residual", (2, 256)), ("sum", (3, 128)), ("y", (4, 256))])
def test_norm_takes_its_rows_shapes_alone(ep, name, shape):
    a = dict(weight=torch.zeros(256), residual=torch.zeros(3, 256), sum=torch.zeros(3, 256), y=torch.zeros(3, 256))
    a[name] = torch.zeros(*shape)
    with pytest.raises(ValueError, match="%s must be \\[" % name):
        ep.ep_rmsnorm(torch.zeros(3, 256), **a)


@pytest.mark.parametrize("name,shape", [("grad_y", (2, 256)), ("weight", (128,)), ("grad_sum", (3, 128)), ("grad_h", (4, 256)), ("grad_weight", (255,))])
def test_norm_gradient_takes_its_rows_shapes_alone(ep, name, shape):
    a = dict(grad_y=torch.zeros(3, 256), weight=torch.zeros(256), grad_sum=torch.zeros(3, 256), grad_h=torch.zeros(3, 256),
             grad_weight=torch.zeros(256))
    a[name] = torch.zeros(*shape)
    with pytest.raises(ValueError, match="%s must be \\[" % name):
        ep.ep_rmsnorm_bwd(h=torch.zeros(3, 256), workspace=torch.zeros(1 << 16), **a)


@pytest.mark.parametrize("name,shape", [("gate", (8, 128)), ("w13", (8, 512, 256)), ("s13", (8, 1, 2)), ("w2", (8, 128, 128)), ("s2", (8, 2, 2)),
                                        ("out", (3, 256)), ("topk_weights", (4, 1)), ("topk_idx", (3, 2))])
def test_few_takes_its_shapes_alone(ep, name, shape):
    a = dict(gate=bf16(8, 256), w13=f8(8, 256, 256), s13=torch.zeros(8, 2, 2), w2=f8(8, 256, 128), s2=torch.zeros(8, 2, 1), out=bf16(4, 256),
             topk_idx=torch.zeros(4, 2, dtype=torch.int64), topk_weights=torch.zeros(4, 2))
    a[name] = torch.zeros(*shape).to(a[name].dtype)
    with pytest.raises(ValueError, match="%s must be \\[" % name):
        ep.ep_moe_few(bf16(4, 256), workspace=torch.zeros(1 << 22), **a)
