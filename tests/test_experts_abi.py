"""Expert products, 4-bit products and router without a GPU: what the C ABI
and the binding refuse, before any launch."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def ep():
    from combine_ep_prepare_gb300 import build
    build.build()
    import combine_ep_prepare_gb300 as ep
    return ep


@pytest.fixture(scope="module")
def handle(ep):
    from combine_ep_prepare_gb300._libep import Handle
    return Handle(ep.ep_register_layer(8, 2, 64, 16, 4)[0], 1 << 20)


P = 4096  # an aligned address that a refused call never follows


def refused(ep, rc, code, word):
    assert rc == code and word in ep.ep_last_error(), (rc, ep.ep_last_error())


def test_products_refuse(ep, handle):
    lib = ep.lib()
    before = ep.ep_launch_count()
    refused(ep, lib.ep_expert_gemm(handle, P, P, 12, 64, P, None), 2, "out_features")
    refused(ep, lib.ep_expert_gemm(handle, P, P, 64, 0, P, None), 2, "in_features")
    refused(ep, lib.ep_expert_gemm(handle, P, P, 64, (1 << 20) + 8, P, None), 2, "in_features")
    refused(ep, lib.ep_expert_gemm(handle, None, P, 64, 64, P, None), 1, "x is NULL")
    refused(ep, lib.ep_expert_gemm(handle, P, P + 8, 64, 64, P, None), 1, "w is not 16-byte aligned")
    refused(ep, lib.ep_expert_gemm(handle, P, P, 64, 64, None, None), 1, "y is NULL")
    refused(ep, lib.ep_expert_gemm_swiglu(handle, P, P, 4, 64, None, P, None), 2, "ffn_features")
    refused(ep, lib.ep_expert_gemm_swiglu(handle, P, P, 64, 64, P + 2, P, None), 1, "pre is not")
    refused(ep, lib.ep_expert_gemm_swiglu(handle, P, P, 64, 64, None, None, None), 1, "act is NULL")
    refused(ep, lib.ep_expert_dgrad(handle, P, None, 64, 64, P, None), 1, "w is NULL")
    refused(ep, lib.ep_expert_dgrad(handle, P, P, 64, -8, P, None), 2, "in_features")
    refused(ep, lib.ep_expert_dgrad_swiglu(handle, P, P, None, 64, 64, P, None), 1, "pre is NULL")
    refused(ep, lib.ep_expert_dgrad_swiglu(handle, P, P, P, 64, 64, P + 4, None), 1, "dpre is not")
    refused(ep, lib.ep_expert_wgrad(handle, P, P, 64, 64, P, 1, 0, None), 1, "dw_dtype")
    refused(ep, lib.ep_expert_wgrad(handle, P, P, 64, 64, P, 0, 2, None), 1, "accumulate")
    refused(ep, lib.ep_expert_wgrad(handle, P, P, 64, 64, None, 2, 1, None), 1, "dw is NULL")
    assert ep.ep_launch_count() == before


def test_w4_refuses(ep, handle):
    lib = ep.lib()
    before = ep.ep_launch_count()
    refused(ep, lib.ep_expert_gemv_w4(handle, P, P, P, 64, 64, 48, P, None), 1, "group")
    refused(ep, lib.ep_expert_gemv_w4(handle, P, P, P, 64, 96, 64, P, None), 2, "multiple of the group")
    refused(ep, lib.ep_expert_gemv_w4(handle, P, P + 1, P, 64, 64, 32, P, None), 1, "wq is not")
    refused(ep, lib.ep_expert_gemv_w4(handle, P, P, P + 1, 64, 64, 32, P, None), 1, "scales is not")
    refused(ep, lib.ep_expert_gemv_w4_swiglu(handle, P, P, P, 4, 64, 32, P, None), 2, "out_features")
    refused(ep, lib.ep_expert_gemv_w4_swiglu(handle, P, P, None, 64, 64, 32, P, None), 1, "scales is NULL")
    from combine_ep_prepare_gb300._libep import Handle
    f32 = Handle(ep.ep_register_layer(8, 2, 64, 16, 4, dtype="fp32")[0], 1 << 20)
    refused(ep, lib.ep_expert_gemv_w4(f32, P, P, P, 64, 64, 32, P, None), 1, "bf16 and fp16")
    assert ep.ep_launch_count() == before


def test_handles_refused(ep):
    from combine_ep_prepare_gb300._libep import Handle
    lib = ep.lib()
    assert lib.ep_expert_gemm(Handle(10 ** 9, P), P, P, 64, 64, P, None) == 5
    assert lib.ep_expert_gemm(Handle(ep.ep_register_layer(8, 2, 64, 16)[0], None), P, P, 64, 64, P, None) == 1
    rm = Handle(ep.ep_register_layer_rank_major(8, 2, 64, 16, 2, 0)[0], 1 << 20)
    refused(ep, lib.ep_expert_gemm(rm, P, P, 64, 64, P, None), 1, "rank-major")
    refused(ep, lib.ep_expert_gemv_w4(rm, P, P, P, 64, 64, 32, P, None), 1, "rank-major")


@pytest.mark.parametrize("change,code,word", [
    (dict(num_experts=0), 6, "num_experts"), (dict(num_experts=1025), 6, "num_experts"),
    (dict(top_k=0), 6, "top_k"), (dict(top_k=33), 6, "top_k"), (dict(num_experts=4, top_k=5), 6, "top_k"),
    (dict(num_groups=3), 6, "num_groups"), (dict(num_groups=64), 6, "num_groups"), (dict(num_groups=0), 6, "num_groups"),
    (dict(num_groups=4, topk_groups=5), 1, "topk_groups"), (dict(topk_groups=0), 1, "topk_groups"),
    (dict(score=2), 1, "score"), (dict(normalize=2), 1, "normalize"), (dict(dtype=3), 1, "dtype"),
    (dict(scale=float("inf")), 1, "scale"), (dict(scale=float("nan")), 1, "scale")])
def test_router_config_refused(ep, change, code, word):
    from combine_ep_prepare_gb300._libep import RouterConfig
    base = dict(num_experts=64, top_k=2, num_groups=1, topk_groups=1, score=0, normalize=1, dtype=2, scale=1.0)
    base.update(change)
    refused(ep, ep.lib().ep_router(RouterConfig(**base), P, None, 4, P, P, None), code, word)
    refused(ep, ep.lib().ep_router_bwd(RouterConfig(**base), P, P, P, 4, P, None), code, word)


def test_router_arguments_refused(ep):
    from combine_ep_prepare_gb300._libep import RouterConfig
    lib = ep.lib()
    c = RouterConfig(64, 2, 1, 1, 0, 1, 2, 1.0)
    before = ep.ep_launch_count()
    refused(ep, lib.ep_router(c, P, None, -1, P, P, None), 2, "num_tokens")
    refused(ep, lib.ep_router(c, P, None, (1 << 23) + 1, P, P, None), 2, "num_tokens")
    refused(ep, lib.ep_router(c, None, None, 4, P, P, None), 1, "logits is NULL")
    refused(ep, lib.ep_router(c, P, P, 4, P, P, None), 1, "bias")
    refused(ep, lib.ep_router(c, P, None, 4, P + 4, P, None), 1, "topk_idx")
    refused(ep, lib.ep_router(c, P, None, 4, P, None, None), 1, "topk_weights")
    refused(ep, lib.ep_router_bwd(c, P, None, P, 4, P, None), 1, "topk_idx")
    refused(ep, lib.ep_router_bwd(c, P, P, P + 2, 4, P, None), 1, "grad_topk_weights")
    refused(ep, lib.ep_router_bwd(c, P, P, P, 4, None, None), 1, "grad_logits")
    assert ep.ep_launch_count() == before


def test_binding_checks_shapes(ep):
    lid, size = ep.ep_register_layer(8, 2, 64, 16, 4)
    R = ep.ep_recv_capacity(lid)
    h = ep.EpHandle(lid, torch.empty(size, dtype=torch.uint8))
    bf = dict(dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ep.ep_expert_gemm(h, torch.empty(R, 64, **bf), torch.empty(8, 32, 64, **bf), torch.empty(R, 32, **bf))
    with pytest.raises(TypeError, match="bfloat16"):
        ep.ep_expert_gemm(h, torch.empty(R, 64, **bf), torch.empty(8, 32, 64), torch.empty(R, 32, **bf))
    with pytest.raises(TypeError, match="dw"):
        ep.ep_expert_wgrad(h, torch.empty(R, 32, **bf), torch.empty(R, 64, **bf), torch.empty(8, 32, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="softmax or sigmoid"):
        ep.ep_router(torch.empty(4, 8), torch.empty(4, 2, dtype=torch.int64), torch.empty(4, 2), score="relu")
    with pytest.raises(ValueError, match="topk_weights"):
        ep.ep_router(torch.empty(4, 8), torch.empty(4, 2, dtype=torch.int64), torch.empty(4, 3))
    with pytest.raises(ValueError, match="bias"):
        ep.ep_router(torch.empty(4, 8), torch.empty(4, 2, dtype=torch.int64), torch.empty(4, 2), bias=torch.empty(7),
                     score="sigmoid")
    with pytest.raises(ValueError, match="group"):
        ep.pack_w4(torch.zeros(1, 8, 96), 64)


def test_shape_checks_before_any_pointer(ep, monkeypatch):
    """Wrong row counts and widths are named, whatever the device."""
    from combine_ep_prepare_gb300 import _libep
    monkeypatch.setattr(_libep, "_ptr", lambda t, dtype=None, name="": 4096)
    lid, size = ep.ep_register_layer(8, 2, 64, 16, 4)
    R = ep.ep_recv_capacity(lid)
    h = ep.EpHandle(lid, torch.empty(size, dtype=torch.uint8))
    w = torch.empty(8, 32, 64)
    with pytest.raises(ValueError, match="x must be"):
        ep.ep_expert_gemm(h, torch.empty(R - 1, 64), w, torch.empty(R, 32))
    with pytest.raises(ValueError, match="y must be"):
        ep.ep_expert_gemm(h, torch.empty(R, 64), w, torch.empty(R, 40))
    with pytest.raises(ValueError, match="8 experts"):
        ep.ep_expert_gemm(h, torch.empty(R, 64), torch.empty(7, 32, 64), torch.empty(R, 32))
    with pytest.raises(ValueError, match="gate rows"):
        ep.ep_expert_gemm_swiglu(h, torch.empty(R, 64), torch.empty(8, 33, 64), torch.empty(R, 16))
    with pytest.raises(ValueError, match="scales"):
        ep.ep_expert_gemv_w4(h, torch.empty(R, 64), torch.empty(8, 32, 32), torch.empty(8, 16, 2), torch.empty(R, 32))
