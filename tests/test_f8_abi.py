"""8-bit rows and products, the norm and a few tokens' layer without a GPU:
what the C ABI and the binding refuse before any launch, and the packing of
weights."""
import ctypes

import pytest
import torch

P = 4096  # an aligned address that a refused call never follows


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


def refused(ep, rc, code, word):
    assert rc == code and word in ep.ep_last_error(), (rc, ep.ep_last_error())


def test_norm_refuses(ep):
    f = ep.lib().ep_rmsnorm
    before = ep.ep_launch_count()
    refused(ep, f(P, P, P, 4, 12, 0, 1e-6, P, P, None, None, None), 2, "multiple of 8")
    refused(ep, f(P, P, P, 4, 24, 0, 1e-6, P, P, P, P, None), 2, "multiple of 16")
    refused(ep, f(P, P, P, 4, 32768 + 8, 0, 1e-6, P, P, None, None, None), 6, "too long")
    refused(ep, f(P, P, P, -1, 64, 0, 1e-6, P, P, None, None, None), 2, "num_tokens")
    refused(ep, f(P, P, P, 1 << 31, 64, 0, 1e-6, P, P, None, None, None), 2, "num_tokens")
    refused(ep, f(P, P, P, 4, 64, 3, 1e-6, P, P, None, None, None), 1, "dtype")
    refused(ep, f(P, P, P, 4, 64, 0, -1.0, P, P, None, None, None), 1, "eps")
    refused(ep, f(P, P, P, 4, 64, 0, float("nan"), P, P, None, None, None), 1, "eps")
    refused(ep, f(P, P, P, 4, 64, 0, 1e-6, P, P, P, None, None), 1, "q and scales")
    refused(ep, f(P, None, P, 4, 64, 0, 1e-6, P, P, None, None, None), 1, "residual")
    refused(ep, f(P, P, P, 4, 64, 0, 1e-6, None, None, None, None, None), 1, "all NULL")
    refused(ep, f(None, P, P, 4, 64, 0, 1e-6, P, P, None, None, None), 1, "x is NULL")
    refused(ep, f(P, P + 8, P, 4, 64, 0, 1e-6, P, P, None, None, None), 1, "residual is not")
    refused(ep, f(P, P, P, 4, 64, 0, 1e-6, P, P + 2, None, None, None), 1, "y is not")
    refused(ep, f(P, P, P, 4, 64, 0, 1e-6, P, P, P, P + 4, None), 1, "scales is not")
    assert ep.ep_launch_count() == before


def test_norm_gradient_refuses(ep):
    f = ep.lib().ep_rmsnorm_bwd
    refused(ep, f(P, P, P, P, 4, 20, 0, 1e-6, P, P, 0, P, None), 2, "multiple of 8")
    refused(ep, f(P, P, P, P, 4, 64, 0, 1e-6, P, P, 2, P, None), 1, "accumulate")
    refused(ep, f(P, None, P, P, 4, 64, 0, 1e-6, P, P, 0, P, None), 1, "h is NULL")
    refused(ep, f(P, P, P, P + 2, 4, 64, 0, 1e-6, P, P, 0, P, None), 1, "grad_sum is not")
    refused(ep, f(P, P, P, P, 4, 64, 0, 1e-6, P, None, 0, P, None), 1, "grad_weight is NULL")
    refused(ep, f(P, P, P, P, 4, 64, 0, 1e-6, P, P, 0, None, None), 1, "workspace is NULL")
    size = ctypes.c_size_t(0)
    w = ep.lib().ep_rmsnorm_bwd_workspace
    assert w(0, 64, ctypes.byref(size)) == 0 and size.value == 0
    sizes = []
    for T in (1, 100, 1000, 100000):
        assert w(T, 64, ctypes.byref(size)) == 0
        sizes.append(size.value)
    assert sizes == sorted(sizes) and sizes[0] == 256
    refused(ep, w(4, 64, None), 1, "bytes")


def test_rows_and_dispatch_refuse(ep, handle):
    from combine_ep_prepare_gb300._libep import Handle
    lib = ep.lib()
    before = ep.ep_launch_count()
    refused(ep, lib.ep_quantize_rows(P, 4, 24, 0, P, P, None), 2, "multiple of 16")
    refused(ep, lib.ep_quantize_rows(P, 4, (1 << 20) + 16, 0, P, P, None), 6, "too long")
    refused(ep, lib.ep_quantize_rows(P, -1, 32, 0, P, P, None), 2, "rows")
    refused(ep, lib.ep_quantize_rows(P, 4, 32, 7, P, P, None), 1, "dtype")
    refused(ep, lib.ep_quantize_rows(P, 4, 32, 0, P + 1, P, None), 1, "q is not")
    refused(ep, lib.ep_quantize_rows(P, 4, 32, 0, P, None, None), 1, "scales is NULL")
    refused(ep, lib.ep_expert_quantize(handle, P, 8, P, P, None), 2, "features")
    refused(ep, lib.ep_expert_quantize(handle, None, 64, P, P, None), 1, "x is NULL")
    f32 = Handle(ep.ep_register_layer(8, 2, 64, 16, 4, dtype="fp32")[0], 1 << 20)
    refused(ep, lib.ep_expert_quantize(f32, P, 64, P, P, None), 1, "bf16 and fp16")
    refused(ep, lib.ep_dispatch_f8(handle, P, 17, P, P, P, P, P, P, None), 2, "num_tokens")
    refused(ep, lib.ep_dispatch_f8(handle, None, 4, P, P, P, P, P, P, None), 1, "topk_idx")
    refused(ep, lib.ep_dispatch_f8(handle, P, 4, P + 8, P, P, P, P, P, None), 1, "tokens is not")
    refused(ep, lib.ep_dispatch_f8(handle, P, 4, P, P + 4, P, P, P, P, None), 1, "scales is not")
    refused(ep, lib.ep_dispatch_f8(handle, P, 4, P, P, P, P, None, P, None), 1, "recv_scales is NULL")
    odd = Handle(ep.ep_register_layer(8, 2, 72, 16, 4)[0], 1 << 20)
    refused(ep, lib.ep_dispatch_f8(odd, P, 4, P, P, P, P, P, P, None), 2, "multiple of 16")
    sharded = Handle(ep.ep_register_layer_sharded(8, 2, 64, 16, 2, 0)[0], 1 << 20)
    refused(ep, lib.ep_dispatch_f8(sharded, P, 4, P, P, P, P, P, P, None), 1, "sharded")
    assert ep.ep_launch_count() == before


def test_products_refuse(ep, handle):
    from combine_ep_prepare_gb300._libep import Handle
    lib = ep.lib()
    before = ep.ep_launch_count()
    refused(ep, lib.ep_expert_gemm_f8(handle, P, P, P, P, 24, 64, P, None), 2, "out_features")
    refused(ep, lib.ep_expert_gemm_f8(handle, P, P, P, P, 64, (1 << 20) + 16, P, None), 2, "in_features")
    refused(ep, lib.ep_expert_gemm_f8(handle, P + 8, P, P, P, 64, 64, P, None), 1, "x is not")
    refused(ep, lib.ep_expert_gemm_f8(handle, P, P + 4, P, P, 64, 64, P, None), 1, "x_scales is not")
    refused(ep, lib.ep_expert_gemm_f8(handle, P, P, P, None, 64, 64, P, None), 1, "w_scales is NULL")
    refused(ep, lib.ep_expert_gemm_f8(handle, P, P, P, P, 64, 64, None, None), 1, "y is NULL")
    refused(ep, lib.ep_expert_gemm_f8_swiglu(handle, P, P, P, P, 64, 64, P, P, P, P, None), 2, "multiple of 128")
    refused(ep, lib.ep_expert_gemm_f8_swiglu(handle, P, P, P, P, 128, 64, None, None, None, None, None), 1, "all NULL")
    refused(ep, lib.ep_expert_gemm_f8_swiglu(handle, P, P, P, P, 128, 64, None, P, P, None, None), 1, "act_q and act_scales")
    refused(ep, lib.ep_expert_dgrad_f8(handle, P, P, None, P, 64, 64, P, None), 1, "w is NULL")
    refused(ep, lib.ep_expert_dgrad_f8(handle, P, P, P, P, 64, 40, P, None), 2, "in_features")
    refused(ep, lib.ep_expert_dgrad_f8_swiglu(handle, P, P, P, P, P, 64, 64, P, None), 2, "multiple of 128")
    refused(ep, lib.ep_expert_dgrad_f8_swiglu(handle, P, P, P, P, None, 64, 128, P, None), 1, "pre is NULL")
    f32 = Handle(ep.ep_register_layer(8, 2, 64, 16, 4, dtype="fp32")[0], 1 << 20)
    refused(ep, lib.ep_expert_gemm_f8(f32, P, P, P, P, 64, 64, P, None), 1, "bf16 and fp16")
    rm = Handle(ep.ep_register_layer_rank_major(8, 2, 64, 16, 2, 0)[0], 1 << 20)
    refused(ep, lib.ep_expert_gemm_f8(rm, P, P, P, P, 64, 64, P, None), 1, "rank-major")
    assert lib.ep_expert_gemm_f8(Handle(10 ** 9, P), P, P, P, P, 64, 64, P, None) == 5
    assert ep.ep_launch_count() == before


def few_config(**change):
    from combine_ep_prepare_gb300._libep import MoeFewConfig, RouterConfig
    r = dict(num_experts=8, top_k=2, num_groups=1, topk_groups=1, score=0, normalize=1, dtype=0, scale=1.0)
    c = dict(hidden=64, ffn=128, dtype=0, weight_f8=0)
    for k, v in change.items():
        (r if k in r and k != "dtype" or k == "gate_dtype" else c)["dtype" if k == "gate_dtype" else k] = v
    return MoeFewConfig(RouterConfig(**r), **c)


@pytest.mark.parametrize("change,code,word", [
    (dict(num_experts=1025), 6, "num_experts"), (dict(top_k=9), 6, "top_k"), (dict(num_groups=3), 6, "num_groups"),
    (dict(score=2), 1, "score"), (dict(gate_dtype=3), 1, "dtype"), (dict(dtype=2), 1, "bf16 and fp16"),
    (dict(weight_f8=2), 1, "weight_f8"), (dict(hidden=12), 2, "hidden"), (dict(hidden=32768 + 8), 2, "hidden"),
    (dict(ffn=4), 2, "ffn"), (dict(weight_f8=1, hidden=72), 2, "hidden"), (dict(weight_f8=1, ffn=64), 2, "ffn")])
def test_few_config_refused(ep, change, code, word):
    size = ctypes.c_size_t(0)
    c = few_config(**change)
    refused(ep, ep.lib().ep_moe_few_workspace(c, 4, ctypes.byref(size)), code, word)
    s = P if change.get("weight_f8") == 1 else None
    refused(ep, ep.lib().ep_moe_few(c, P, P, None, P, s, P, s, 4, P, P, P, P, None), code, word)


def test_few_arguments_refused(ep):
    f = ep.lib().ep_moe_few
    c, c8, sig = few_config(), few_config(weight_f8=1), few_config(score=1)
    before = ep.ep_launch_count()
    refused(ep, f(c, P, P, None, P, None, P, None, 33, P, P, P, P, None), 2, "num_tokens")
    refused(ep, f(c, P, P, None, P, None, P, None, -1, P, P, P, P, None), 2, "num_tokens")
    refused(ep, f(c, P, P, P, P, None, P, None, 4, P, P, P, P, None), 1, "bias")
    refused(ep, f(sig, P, P, P + 2, P, None, P, None, 4, P, P, P, P, None), 1, "bias is not")
    refused(ep, f(c, P, P, None, P, P, P, P, 4, P, P, P, P, None), 1, "8-bit weights")
    refused(ep, f(c8, P, P, None, P, None, P, P, 4, P, P, P, P, None), 1, "w13_scales is NULL")
    refused(ep, f(c, None, P, None, P, None, P, None, 4, P, P, P, P, None), 1, "x is NULL")
    refused(ep, f(c, P, P + 8, None, P, None, P, None, 4, P, P, P, P, None), 1, "gate is not")
    refused(ep, f(c, P, P, None, P, None, None, None, 4, P, P, P, P, None), 1, "w2 is NULL")
    refused(ep, f(c, P, P, None, P, None, P, None, 4, P, P + 4, P, P, None), 1, "topk_idx is not")
    refused(ep, f(c, P, P, None, P, None, P, None, 4, P, P, P, P + 128, None), 1, "workspace is not")
    assert ep.ep_launch_count() == before


def test_few_workspace_covers_smaller_batches_and_both_types(ep):
    size = ctypes.c_size_t(0)
    got = []
    for T in (0, 1, 5, 32):
        for f8 in (0, 1):
            assert ep.lib().ep_moe_few_workspace(few_config(weight_f8=f8), T, ctypes.byref(size)) == 0
            got.append(size.value)
    assert got[1::2] == sorted(got[1::2]) and all(a <= b for a, b in zip(got[0::2], got[1::2]))


def test_binding_checks(ep):
    lid, size = ep.ep_register_layer(8, 2, 64, 16, 4)
    R = ep.ep_recv_capacity(lid)
    h = ep.EpHandle(lid, torch.empty(size, dtype=torch.uint8))
    f8 = torch.float8_e4m3fn
    rows, scales = torch.empty(R, 64, dtype=f8), torch.empty(R, 4)
    with pytest.raises(ValueError, match="w_scales|CUDA"):
        ep.ep_expert_gemm_f8(h, rows, scales, torch.empty(8, 32, 64, dtype=f8), torch.empty(8, 1, 2), torch.empty(R, 32))
    with pytest.raises(TypeError, match="float8"):
        ep.ep_expert_gemm_f8(h, rows, scales, torch.empty(8, 32, 64), torch.empty(8, 1, 1), torch.empty(R, 32))
    with pytest.raises(ValueError, match="CUDA|scales must be"):
        ep.ep_quantize_rows(torch.empty(3, 256), torch.empty(3, 256, dtype=f8), torch.empty(3, 2))
    with pytest.raises(ValueError, match="workspace must hold"):
        ep.ep_rmsnorm_bwd(*[torch.empty(3, 64)] * 2, torch.empty(64), torch.empty(3, 64), torch.empty(64), torch.empty(4))
    with pytest.raises(ValueError, match="need s13"):
        ep.ep_moe_few(torch.empty(2, 64, dtype=torch.bfloat16), torch.empty(8, 64), torch.empty(8, 256, 64, dtype=f8),
                      torch.empty(8, 64, 128, dtype=f8), torch.empty(2, 64), torch.empty(2, 2, dtype=torch.int64), torch.empty(2, 2),
                      torch.empty(1 << 20, dtype=torch.uint8))
    assert [ep.scale_columns(n) for n in (16, 128, 512, 528, 7168)] == [4, 4, 4, 8, 56]


@pytest.mark.parametrize("n,k", [(128, 128), (16, 16), (272, 400), (130, 48)])
def test_pack_f8(ep, n, k):
    g = torch.Generator().manual_seed(3)
    w = torch.randn(2, n, k, generator=g) * torch.logspace(-3, 3, k)
    w[1, : min(n, 128), : min(k, 128)] = 0  # a block of zeros
    q, s = ep.pack_f8(w)
    assert q.shape == w.shape and s.shape == (2, (n + 127) // 128, (k + 127) // 128) and bool(torch.isfinite(s).all())
    scale = s.repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k].double()
    back = q.double() * scale
    # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale below its normal range; float32's two roundings beside it
    assert bool(((back - w.double()).abs() <= w.double().abs() * (2.0 ** -4 + 2.0 ** -22) + scale * 2.0 ** -10).all())
    assert bool((back[1, : min(n, 128), : min(k, 128)] == 0).all())
