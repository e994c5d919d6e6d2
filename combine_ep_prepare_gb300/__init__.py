"""combine_ep_prepare_gb300 -- MoE expert-parallel dispatch / combine on one
GB300, as hand-written sm_103a CUDA kernels behind a C ABI (libep).

    import combine_ep_prepare_gb300 as ep
    lid, size = ep.ep_register_layer(num_experts=E, top_k=K, hidden=H, max_tokens=T)
    h = ep.alloc_handle(lid, size)
    ep.ep_prepare(h, topk_idx, token_counts, alignment)
    ep.ep_dispatch(h, topk_idx, tokens, topk_weights, recv_tokens, recv_topk_weights)
    ep.ep_expert_gemm_swiglu(h, recv_tokens, w13, act)
    ep.ep_expert_gemm(h, act, w2, expert_out)
    ep.ep_combine_weighted(h, expert_out, recv_topk_weights, result)

``moe_layer`` runs a whole layer on these calls.

The binding (``_libep``) is loaded on first use of an ``ep_*`` name, and
raises ImportError when libep.so has not been built: there is no CPU path.
``workloads`` (seeded synthetic inputs) imports without the library.
"""
from . import workloads  # noqa: F401

_BINDING_NAMES = {
    "EpError", "EpHandle", "alloc_handle", "lib", "SYMBOLS",
    "EP_ST_BAD_INDEX", "EP_ST_OVERFLOW", "EP_ST_TOKENS_MISMATCH", "EP_ST_NOT_PREPARED",
    "ep_abi_version", "ep_last_error", "ep_launch_count", "ep_register_layer",
    "ep_recv_capacity", "ep_prepare", "ep_prepare_static_scratch", "ep_dispatch", "ep_combine", "ep_dispatch_bwd",
    "ep_combine_bwd", "ep_combine_weighted", "ep_combine_weighted_bwd", "ep_expert_offsets", "ep_token_slots", "ep_read_info",
    "EP_ST_COUNTS_MISMATCH", "EP_ST_BAD_POINTER", "EP_ST_TIMEOUT", "ep_register_layer_sharded", "pointer_table",
    "ep_shard_count", "exchange_counts", "ep_shard_prepare", "ep_shard_dispatch", "ep_shard_combine",
    "ep_shard_combine_bwd", "ep_shard_dispatch_bwd", "ep_shard_token_owners",
    "ep_register_layer_rank_major", "ep_rank_major_count", "ep_rank_major_prepare",
    "ep_rank_major_dispatch", "ep_rank_major_combine", "ep_rank_major_combine_bwd",
    "ep_rank_major_dispatch_bwd",
    "ep_expert_gemm", "ep_expert_gemm_swiglu", "ep_expert_dgrad", "ep_expert_dgrad_swiglu", "ep_expert_wgrad",
    "ep_expert_gemv_w4", "ep_expert_gemv_w4_swiglu", "pack_w4", "ep_router", "ep_router_bwd",
    "ep_rmsnorm", "rmsnorm_bwd_workspace", "ep_rmsnorm_bwd", "ep_quantize_rows", "ep_expert_quantize", "ep_dispatch_f8",
    "ep_expert_gemm_f8", "ep_expert_gemm_f8_swiglu", "ep_expert_dgrad_f8", "ep_expert_dgrad_f8_swiglu", "pack_f8",
    "scale_columns", "ep_moe_few", "moe_few_workspace", "MAX_FEW_TOKENS",
}


def __getattr__(name):
    if name in _BINDING_NAMES:
        from . import _libep
        value = getattr(_libep, name)
        globals()[name] = value  # later uses find it without this call
        return value
    raise AttributeError(name)
