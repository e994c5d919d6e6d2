"""ctypes binding of libep (include/ep.h).

Argument marshalling only: tensors become device pointers and sizes, the
current torch stream becomes a cudaStream_t, status codes become
exceptions.  Every step of the path runs in libep's CUDA kernels; there is no
fallback, and importing this module fails loudly when libep.so is missing.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from .build import library_path

EP_OK = 0
EP_ST_BAD_INDEX = 1
EP_ST_OVERFLOW = 2
EP_ST_TOKENS_MISMATCH = 4
EP_ST_NOT_PREPARED = 8
EP_ST_COUNTS_MISMATCH = 16
EP_ST_BAD_POINTER = 32
EP_ST_TIMEOUT = 64
ERROR_NAMES = {1: "EP_ERR_INVALID_ARG", 2: "EP_ERR_SHAPE", 3: "EP_ERR_UNSUPPORTED_ARCH",
               4: "EP_ERR_CUDA", 5: "EP_ERR_NOT_REGISTERED", 6: "EP_ERR_LIMIT"}


class EpError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__("%s: %s" % (ERROR_NAMES.get(code, str(code)), message))
        self.code = code


class LayerConfig(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int64), ("top_k", ctypes.c_int64),
                ("hidden", ctypes.c_int64), ("max_tokens", ctypes.c_int64),
                ("max_alignment", ctypes.c_int64), ("recv_capacity", ctypes.c_int64),
                ("dtype", ctypes.c_int64)]


# Payload element types (ep_dtype_t) and the torch dtype of each.
DTYPE_CODES = {"bf16": 0, "fp16": 1, "fp32": 2}
TORCH_DTYPES = {0: torch.bfloat16, 1: torch.float16, 2: torch.float32}
_layer_dtype = {}  # layer id -> torch dtype of its payload rows
_layer_experts = {}  # layer id -> (experts whose rows this rank holds, receive capacity)


class RouterConfig(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int64), ("top_k", ctypes.c_int64),
                ("num_groups", ctypes.c_int64), ("topk_groups", ctypes.c_int64),
                ("score", ctypes.c_int64), ("normalize", ctypes.c_int64),
                ("dtype", ctypes.c_int64), ("scale", ctypes.c_float)]


SCORE_CODES = {"softmax": 0, "sigmoid": 1}


class Handle(ctypes.Structure):
    _fields_ = [("id", ctypes.c_uint64), ("mem", ctypes.c_void_p)]


class Info(ctypes.Structure):
    _fields_ = [("status", ctypes.c_uint32), ("num_tokens", ctypes.c_int32),
                ("used_rows", ctypes.c_int32), ("padding_rows", ctypes.c_int32)]


def _load(path=None):
    path = path or library_path()
    if not os.path.exists(path):
        raise ImportError("libep.so is not built (%s); run __graft_entry__.build() "
                          "or python -m combine_ep_prepare_gb300.build" % path)
    lib = ctypes.CDLL(path)
    u64, i64, p, st = ctypes.c_uint64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    sig = {
        "ep_abi_version": ([], ctypes.c_uint32),
        "ep_last_error": ([], ctypes.c_char_p),
        "ep_launch_count": ([], ctypes.c_uint64),
        "ep_register_layer": ([LayerConfig, ctypes.POINTER(u64), ctypes.POINTER(ctypes.c_size_t)], st),
        "ep_recv_capacity": ([u64, ctypes.POINTER(i64)], st),
        "ep_prepare": ([Handle, p, i64, p, i64, p], st),
        "ep_prepare_static_scratch": ([Handle, p, i64, p, i64, p], st),
        "ep_dispatch": ([Handle, p, i64, p, p, p, p, p], st),
        "ep_combine": ([Handle, p, i64, p, p], st),
        "ep_dispatch_bwd": ([Handle, p, p, i64, p, p, p], st),
        "ep_combine_bwd": ([Handle, p, i64, p, p], st),
        "ep_combine_weighted": ([Handle, p, p, i64, p, p], st),
        "ep_combine_weighted_bwd": ([Handle, p, p, p, i64, p, p, p], st),
        "ep_expert_offsets": ([Handle, p, p], st),
        "ep_token_slots": ([Handle, p, i64, p], st),
        "ep_read_info": ([Handle, ctypes.POINTER(Info), p], st),
        "ep_register_layer_sharded": ([LayerConfig, i64, i64, ctypes.POINTER(u64),
                                       ctypes.POINTER(ctypes.c_size_t)], st),
        "ep_shard_count": ([Handle, p, i64, p, p], st),
        "ep_shard_prepare": ([Handle, p, i64, p, p, i64, p], st),
        "ep_shard_dispatch": ([Handle, i64, p, p, p, p, p], st),
        "ep_shard_combine": ([Handle, p, i64, p, p], st),
        "ep_shard_combine_bwd": ([Handle, p, i64, p, p], st),
        "ep_shard_dispatch_bwd": ([Handle, p, p, i64, p, p, p], st),
        "ep_shard_token_owners": ([Handle, p, i64, p], st),
        "ep_register_layer_rank_major": ([LayerConfig, i64, i64, ctypes.POINTER(u64),
                                          ctypes.POINTER(ctypes.c_size_t)], st),
        "ep_rank_major_count": ([Handle, p, i64, p, p], st),
        "ep_rank_major_prepare": ([Handle, p, i64, p, p, p], st),
        "ep_rank_major_dispatch": ([Handle, p, i64, p, p, p, p, p, p], st),
        "ep_rank_major_combine": ([Handle, p, i64, p, p], st),
        "ep_rank_major_combine_bwd": ([Handle, p, i64, p, p], st),
        "ep_rank_major_dispatch_bwd": ([Handle, p, p, i64, p, p, p], st),
        "ep_expert_gemm": ([Handle, p, p, i64, i64, p, p], st),
        "ep_expert_gemm_swiglu": ([Handle, p, p, i64, i64, p, p, p], st),
        "ep_expert_dgrad": ([Handle, p, p, i64, i64, p, p], st),
        "ep_expert_dgrad_swiglu": ([Handle, p, p, p, i64, i64, p, p], st),
        "ep_expert_wgrad": ([Handle, p, p, i64, i64, p, i64, ctypes.c_int, p], st),
        "ep_expert_gemv_w4": ([Handle, p, p, p, i64, i64, i64, p, p], st),
        "ep_expert_gemv_w4_swiglu": ([Handle, p, p, p, i64, i64, i64, p, p], st),
        "ep_router": ([RouterConfig, p, p, i64, p, p, p], st),
        "ep_router_bwd": ([RouterConfig, p, p, p, i64, p, p], st),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()
SYMBOLS = ("ep_abi_version", "ep_last_error", "ep_launch_count", "ep_register_layer",
           "ep_recv_capacity", "ep_prepare", "ep_prepare_static_scratch", "ep_dispatch", "ep_combine", "ep_dispatch_bwd",
           "ep_combine_bwd", "ep_combine_weighted", "ep_combine_weighted_bwd", "ep_expert_offsets", "ep_token_slots", "ep_read_info",
           "ep_register_layer_sharded", "ep_shard_count", "ep_shard_prepare", "ep_shard_dispatch",
           "ep_shard_combine", "ep_shard_combine_bwd", "ep_shard_dispatch_bwd", "ep_shard_token_owners",
           "ep_register_layer_rank_major", "ep_rank_major_count", "ep_rank_major_prepare",
           "ep_rank_major_dispatch", "ep_rank_major_combine", "ep_rank_major_combine_bwd",
           "ep_rank_major_dispatch_bwd",
           "ep_expert_gemm", "ep_expert_gemm_swiglu", "ep_expert_dgrad", "ep_expert_dgrad_swiglu",
           "ep_expert_wgrad", "ep_expert_gemv_w4", "ep_expert_gemv_w4_swiglu", "ep_router", "ep_router_bwd")


def lib():
    return _lib


def _check(code: int):
    if code != EP_OK:
        raise EpError(code, _lib.ep_last_error().decode())


# The current stream's handle without a Stream object: building one costs more
# than a small kernel takes.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None and _raw_device is not None and torch.cuda.is_initialized():
            return _raw_stream(_raw_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t: Optional[torch.Tensor], dtype=None, name="tensor") -> Optional[int]:
    if t is None:
        return None
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t.data_ptr() or None


class EpHandle:
    """A registered layer id plus the caller-owned handle memory of one
    in-flight step (TransformerEngine's NVTEEpHandle {id, mem})."""

    def __init__(self, layer_id: int, mem: torch.Tensor):
        self.id = int(layer_id)
        self.mem = mem

    @property
    def c(self) -> Handle:
        return Handle(self.id, self.mem.data_ptr())


def ep_abi_version() -> int:
    return int(_lib.ep_abi_version())


def ep_last_error() -> str:
    return _lib.ep_last_error().decode()


def ep_launch_count() -> int:
    return int(_lib.ep_launch_count())


_DTYPE_NAMES = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}


def _dtype_code(dtype) -> int:
    if not isinstance(dtype, str):
        dtype = _DTYPE_NAMES.get(dtype, str(dtype))
    if dtype not in DTYPE_CODES:
        raise TypeError("payload dtype must be bf16, fp16 or fp32, got %s" % dtype)
    return DTYPE_CODES[dtype]


def ep_register_layer(num_experts: int, top_k: int, hidden: int, max_tokens: int,
                      max_alignment: int = 128, recv_capacity: int = 0, dtype="bf16"):
    """Returns (layer_id, handle_mem_size_bytes).  dtype: "bf16", "fp16",
    "fp32" or the matching torch dtype."""
    code = _dtype_code(dtype)
    cfg = LayerConfig(num_experts, top_k, hidden, max_tokens, max_alignment, recv_capacity, code)
    lid = ctypes.c_uint64(0)
    size = ctypes.c_size_t(0)
    _check(_lib.ep_register_layer(cfg, ctypes.byref(lid), ctypes.byref(size)))
    _layer_dtype[int(lid.value)] = TORCH_DTYPES[code]
    _layer_experts[int(lid.value)] = (num_experts, ep_recv_capacity(int(lid.value)))
    return int(lid.value), int(size.value)


def ep_register_layer_sharded(num_experts: int, top_k: int, hidden: int, max_tokens: int,
                              num_ranks: int, rank: int, max_alignment: int = 128,
                              recv_capacity: int = 0, dtype="bf16"):
    """A layer of rank `rank` of `num_ranks` (expert parallelism): rank q
    owns experts [q*E/N, (q+1)*E/N).  max_tokens is the largest batch of any
    rank.  Returns (layer_id, handle_mem_size_bytes)."""
    code = _dtype_code(dtype)
    cfg = LayerConfig(num_experts, top_k, hidden, max_tokens, max_alignment, recv_capacity, code)
    lid = ctypes.c_uint64(0)
    size = ctypes.c_size_t(0)
    _check(_lib.ep_register_layer_sharded(cfg, num_ranks, rank, ctypes.byref(lid), ctypes.byref(size)))
    _layer_dtype[int(lid.value)] = TORCH_DTYPES[code]
    _layer_experts[int(lid.value)] = (num_experts // num_ranks, ep_recv_capacity(int(lid.value)))
    return int(lid.value), int(size.value)


def _payload(h) -> "torch.dtype":
    return _layer_dtype.get(h.id, torch.bfloat16)


def ep_recv_capacity(layer_id: int) -> int:
    rows = ctypes.c_int64(0)
    _check(_lib.ep_recv_capacity(layer_id, ctypes.byref(rows)))
    return int(rows.value)


def alloc_handle(layer_id: int, size: int, device="cuda") -> EpHandle:
    """Convenience: allocate handle memory (once, outside the step) with torch,
    zero-filled, so that memory the caching allocator hands back from an
    earlier handle cannot pass for a prepared one."""
    return EpHandle(layer_id, torch.zeros(size, dtype=torch.uint8, device=device))


def ep_prepare(h: EpHandle, topk_idx: torch.Tensor, token_counts: torch.Tensor,
               alignment: int, stream=None):
    T = topk_idx.shape[0]
    _check(_lib.ep_prepare(h.c, _ptr(topk_idx, torch.int64, "topk_idx"), T,
                           _ptr(token_counts, torch.int32, "token_counts"), alignment,
                           _stream(stream)))


def ep_prepare_static_scratch(h: EpHandle, topk_idx: torch.Tensor, token_counts: torch.Tensor,
                              alignment: int, stream=None):
    """ep_prepare without any scratch from the caller: for code that cannot
    allocate device memory (see include/ep.h)."""
    T = topk_idx.shape[0]
    _check(_lib.ep_prepare_static_scratch(h.c, _ptr(topk_idx, torch.int64, "topk_idx"), T,
                                          _ptr(token_counts, torch.int32, "token_counts"),
                                          alignment, _stream(stream)))


def ep_dispatch(h: EpHandle, topk_idx: torch.Tensor, tokens: torch.Tensor,
                topk_weights: torch.Tensor, recv_tokens: torch.Tensor,
                recv_topk_weights: torch.Tensor, stream=None):
    T = tokens.shape[0]
    _check(_lib.ep_dispatch(h.c, _ptr(topk_idx, torch.int64, "topk_idx"), T,
                            _ptr(tokens, _payload(h), "tokens"),
                            _ptr(topk_weights, torch.float32, "topk_weights"),
                            _ptr(recv_tokens, _payload(h), "recv_tokens"),
                            _ptr(recv_topk_weights, torch.float32, "recv_topk_weights"),
                            _stream(stream)))


def ep_combine(h: EpHandle, expert_out: torch.Tensor, result: torch.Tensor, stream=None):
    T = result.shape[0]
    _check(_lib.ep_combine(h.c, _ptr(expert_out, _payload(h), "expert_out"), T,
                           _ptr(result, _payload(h), "result"), _stream(stream)))


def ep_dispatch_bwd(h: EpHandle, grad: torch.Tensor, g_recv_topk_weights: Optional[torch.Tensor],
                    grad_tokens: torch.Tensor, grad_topk_weights: torch.Tensor, stream=None):
    T = grad_tokens.shape[0]
    _check(_lib.ep_dispatch_bwd(h.c, _ptr(grad, _payload(h), "grad"),
                                _ptr(g_recv_topk_weights, torch.float32, "g_recv_topk_weights"), T,
                                _ptr(grad_tokens, _payload(h), "grad_tokens"),
                                _ptr(grad_topk_weights, torch.float32, "grad_topk_weights"),
                                _stream(stream)))


def ep_combine_bwd(h: EpHandle, grad: torch.Tensor, grad_expert_out: torch.Tensor, stream=None):
    T = grad.shape[0]
    _check(_lib.ep_combine_bwd(h.c, _ptr(grad, _payload(h), "grad"), T,
                               _ptr(grad_expert_out, _payload(h), "grad_expert_out"),
                               _stream(stream)))


def ep_combine_weighted(h: EpHandle, expert_out: torch.Tensor, recv_topk_weights: torch.Tensor,
                        result: torch.Tensor, stream=None):
    T = result.shape[0]
    _check(_lib.ep_combine_weighted(h.c, _ptr(expert_out, _payload(h), "expert_out"),
                                    _ptr(recv_topk_weights, torch.float32, "recv_topk_weights"), T,
                                    _ptr(result, _payload(h), "result"), _stream(stream)))


def ep_combine_weighted_bwd(h: EpHandle, grad: torch.Tensor, expert_out: torch.Tensor,
                            recv_topk_weights: torch.Tensor, grad_expert_out: torch.Tensor,
                            g_recv_topk_weights: torch.Tensor, stream=None):
    T = grad.shape[0]
    _check(_lib.ep_combine_weighted_bwd(h.c, _ptr(grad, _payload(h), "grad"),
                                        _ptr(expert_out, _payload(h), "expert_out"),
                                        _ptr(recv_topk_weights, torch.float32, "recv_topk_weights"), T,
                                        _ptr(grad_expert_out, _payload(h), "grad_expert_out"),
                                        _ptr(g_recv_topk_weights, torch.float32, "g_recv_topk_weights"),
                                        _stream(stream)))


def ep_expert_offsets(h: EpHandle, offsets: torch.Tensor, stream=None):
    _check(_lib.ep_expert_offsets(h.c, _ptr(offsets, torch.int32, "offsets"), _stream(stream)))


def ep_token_slots(h: EpHandle, slots: torch.Tensor, stream=None):
    _check(_lib.ep_token_slots(h.c, _ptr(slots, torch.int32, "slots"), slots.shape[0],
                               _stream(stream)))


def ep_read_info(h: EpHandle, stream=None) -> dict:
    info = Info()
    _check(_lib.ep_read_info(h.c, ctypes.byref(info), _stream(stream)))
    return {"status": int(info.status), "num_tokens": int(info.num_tokens),
            "used_rows": int(info.used_rows), "padding_rows": int(info.padding_rows)}


# ----------------------------------------------------------------------------
# Sharded layers (expert parallelism over N ranks)
# ----------------------------------------------------------------------------

def pointer_table(tensors, device=None) -> torch.Tensor:
    """Device array of the tensors' addresses (int64 [N]), for the row calls
    of a sharded layer: entry r = rank r's buffer as this rank's device
    addresses it.  Build it once, outside the step."""
    ptrs = [0 if t is None else t.data_ptr() for t in tensors]
    dev = device if device is not None else next(t.device for t in tensors if t is not None)
    return torch.tensor(ptrs, dtype=torch.int64, device=dev)


def _table(tab: Optional[torch.Tensor], name: str) -> Optional[int]:
    if tab is None:
        return None
    return _ptr(tab, torch.int64, name)


def ep_shard_count(h: EpHandle, topk_idx: torch.Tensor, local_counts: torch.Tensor, stream=None):
    T = topk_idx.shape[0]
    _check(_lib.ep_shard_count(h.c, _ptr(topk_idx, torch.int64, "topk_idx"), T,
                               _ptr(local_counts, torch.int32, "local_counts"), _stream(stream)))


def exchange_counts(local_counts: torch.Tensor, group=None) -> torch.Tensor:
    """All-gather every rank's ep_shard_count output over a
    torch.distributed group: returns int32 [N, E], row r = rank r's counts
    (the routing-table all-gather of the pages' prepare)."""
    import torch.distributed as dist
    n = dist.get_world_size(group)
    flat = local_counts.contiguous().view(-1)
    out = torch.empty(n * flat.numel(), dtype=local_counts.dtype, device=local_counts.device)
    dist.all_gather_into_tensor(out, flat, group=group)
    return out.view((n,) + tuple(local_counts.shape))


def ep_shard_prepare(h: EpHandle, topk_idx: torch.Tensor, all_counts: torch.Tensor,
                     token_counts: torch.Tensor, alignment: int, stream=None):
    T = topk_idx.shape[0]
    _check(_lib.ep_shard_prepare(h.c, _ptr(topk_idx, torch.int64, "topk_idx"), T,
                                 _ptr(all_counts, torch.int32, "all_counts"),
                                 _ptr(token_counts, torch.int32, "token_counts"), alignment,
                                 _stream(stream)))


def ep_shard_dispatch(h: EpHandle, tokens: torch.Tensor, topk_weights: torch.Tensor,
                      recv_tokens: torch.Tensor, recv_topk_weights: torch.Tensor, stream=None):
    """recv_tokens, recv_topk_weights: pointer tables (pointer_table)."""
    T = tokens.shape[0]
    _check(_lib.ep_shard_dispatch(h.c, T, _ptr(tokens, _payload(h), "tokens"),
                                  _ptr(topk_weights, torch.float32, "topk_weights"),
                                  _table(recv_tokens, "recv_tokens"),
                                  _table(recv_topk_weights, "recv_topk_weights"), _stream(stream)))


def ep_shard_combine(h: EpHandle, expert_out: torch.Tensor, result: torch.Tensor, stream=None):
    """expert_out: pointer table."""
    T = result.shape[0]
    _check(_lib.ep_shard_combine(h.c, _table(expert_out, "expert_out"), T,
                                 _ptr(result, _payload(h), "result"), _stream(stream)))


def ep_shard_combine_bwd(h: EpHandle, grad: torch.Tensor, grad_expert_out: torch.Tensor,
                         stream=None):
    """grad_expert_out: pointer table."""
    T = grad.shape[0]
    _check(_lib.ep_shard_combine_bwd(h.c, _ptr(grad, _payload(h), "grad"), T,
                                     _table(grad_expert_out, "grad_expert_out"), _stream(stream)))


def ep_shard_dispatch_bwd(h: EpHandle, grad: torch.Tensor, g_recv_topk_weights: Optional[torch.Tensor],
                          grad_tokens: torch.Tensor, grad_topk_weights: torch.Tensor, stream=None):
    """grad, g_recv_topk_weights: pointer tables (the latter may be None)."""
    T = grad_tokens.shape[0]
    _check(_lib.ep_shard_dispatch_bwd(h.c, _table(grad, "grad"),
                                      _table(g_recv_topk_weights, "g_recv_topk_weights"), T,
                                      _ptr(grad_tokens, _payload(h), "grad_tokens"),
                                      _ptr(grad_topk_weights, torch.float32, "grad_topk_weights"),
                                      _stream(stream)))


def ep_shard_token_owners(h: EpHandle, owners: torch.Tensor, stream=None):
    _check(_lib.ep_shard_token_owners(h.c, _ptr(owners, torch.int32, "owners"), owners.shape[0],
                                      _stream(stream)))


# ----------------------------------------------------------------------------
# Rank-major layers (sharded, at most N * max_tokens received rows per owner;
# the owner permutes them with a single-buffer layer of E/N experts)
# ----------------------------------------------------------------------------

def ep_register_layer_rank_major(num_experts: int, top_k: int, hidden: int, max_tokens: int,
                                 num_ranks: int, rank: int, recv_capacity: int = 0, dtype="bf16"):
    """A rank-major layer of rank `rank` of `num_ranks`.  recv_capacity =
    rows per owner (0: num_ranks * max_tokens).  Returns (layer_id,
    handle_mem_size_bytes)."""
    code = _dtype_code(dtype)
    cfg = LayerConfig(num_experts, top_k, hidden, max_tokens, 1, recv_capacity, code)
    lid = ctypes.c_uint64(0)
    size = ctypes.c_size_t(0)
    _check(_lib.ep_register_layer_rank_major(cfg, num_ranks, rank, ctypes.byref(lid), ctypes.byref(size)))
    _layer_dtype[int(lid.value)] = TORCH_DTYPES[code]
    return int(lid.value), int(size.value)


def ep_rank_major_count(h: EpHandle, topk_idx: torch.Tensor, local_counts: torch.Tensor, stream=None):
    """local_counts: int32 [N], this rank's tokens per owner."""
    T = topk_idx.shape[0]
    _check(_lib.ep_rank_major_count(h.c, _ptr(topk_idx, torch.int64, "topk_idx"), T,
                                    _ptr(local_counts, torch.int32, "local_counts"), _stream(stream)))


def ep_rank_major_prepare(h: EpHandle, topk_idx: torch.Tensor, all_counts: torch.Tensor,
                          recv_rows: torch.Tensor, stream=None):
    """all_counts: int32 [N, N] (exchange_counts of the count call);
    recv_rows: int32 [1], the rows this rank receives."""
    T = topk_idx.shape[0]
    _check(_lib.ep_rank_major_prepare(h.c, _ptr(topk_idx, torch.int64, "topk_idx"), T,
                                      _ptr(all_counts, torch.int32, "all_counts"),
                                      _ptr(recv_rows, torch.int32, "recv_rows"), _stream(stream)))


def ep_rank_major_dispatch(h: EpHandle, topk_idx: torch.Tensor, tokens: torch.Tensor,
                           topk_weights: Optional[torch.Tensor], recv_tokens: torch.Tensor,
                           recv_topk_idx: torch.Tensor, recv_topk_weights: Optional[torch.Tensor],
                           stream=None):
    """recv_tokens, recv_topk_idx, recv_topk_weights: pointer tables (the
    last may be None: ids only)."""
    T = tokens.shape[0]
    _check(_lib.ep_rank_major_dispatch(
        h.c, _ptr(topk_idx, torch.int64, "topk_idx"), T, _ptr(tokens, _payload(h), "tokens"),
        None if topk_weights is None else _ptr(topk_weights, torch.float32, "topk_weights"),
        _table(recv_tokens, "recv_tokens"), _table(recv_topk_idx, "recv_topk_idx"),
        _table(recv_topk_weights, "recv_topk_weights"), _stream(stream)))


def ep_rank_major_combine(h: EpHandle, partial: torch.Tensor, result: torch.Tensor, stream=None):
    """partial: pointer table of the owners' [M_q, H] partial rows."""
    T = result.shape[0]
    _check(_lib.ep_rank_major_combine(h.c, _table(partial, "partial"), T,
                                      _ptr(result, _payload(h), "result"), _stream(stream)))


def ep_rank_major_combine_bwd(h: EpHandle, grad: torch.Tensor, grad_recv: torch.Tensor, stream=None):
    """grad_recv: pointer table."""
    T = grad.shape[0]
    _check(_lib.ep_rank_major_combine_bwd(h.c, _ptr(grad, _payload(h), "grad"), T,
                                          _table(grad_recv, "grad_recv"), _stream(stream)))


def ep_rank_major_dispatch_bwd(h: EpHandle, grad_recv: torch.Tensor,
                               g_recv_topk_weights: Optional[torch.Tensor], grad_tokens: torch.Tensor,
                               grad_topk_weights: torch.Tensor, stream=None):
    """grad_recv, g_recv_topk_weights: pointer tables (the latter may be None)."""
    T = grad_tokens.shape[0]
    _check(_lib.ep_rank_major_dispatch_bwd(h.c, _table(grad_recv, "grad_recv"),
                                           _table(g_recv_topk_weights, "g_recv_topk_weights"), T,
                                           _ptr(grad_tokens, _payload(h), "grad_tokens"),
                                           _ptr(grad_topk_weights, torch.float32, "grad_topk_weights"),
                                           _stream(stream)))


# ----------------------------------------------------------------------------
# Expert products on the receive rows of a prepared handle
# ----------------------------------------------------------------------------

def _rows(h: EpHandle, t: torch.Tensor, width: int, name: str) -> int:
    """A receive-row buffer: at least the layer's capacity of rows of `width`
    payload elements."""
    p = _ptr(t, _payload(h), name)
    capacity = _layer_experts.get(h.id, (0, 0))[1]
    if t.dim() != 2 or t.shape[1] != width or t.shape[0] < capacity:
        raise ValueError("%s must be [>= %d rows, %d], got %s" % (name, capacity, width, tuple(t.shape)))
    return p


def _expert_weights(h: EpHandle, t: torch.Tensor, name: str, dtype=None):
    """A per-expert array [E, n, k]: pointer and the two sizes."""
    p = _ptr(t, dtype if dtype is not None else _payload(h), name)
    experts = _layer_experts.get(h.id, (t.shape[0], 0))[0]
    if t.dim() != 3 or t.shape[0] != experts:
        raise ValueError("%s must be [%d experts, out, in], got %s" % (name, experts, tuple(t.shape)))
    return p, t.shape[1], t.shape[2]


def _gated(n: int, name: str) -> int:
    if n % 2:
        raise ValueError("%s must hold as many gate rows as up rows, got %d" % (name, n))
    return n // 2


def ep_expert_gemm(h: EpHandle, x: torch.Tensor, w: torch.Tensor, y: torch.Tensor, stream=None):
    """y[r] = w[e] x[r] for the rows of each expert e; w [E, out, in]."""
    wp, n, k = _expert_weights(h, w, "w")
    _check(_lib.ep_expert_gemm(h.c, _rows(h, x, k, "x"), wp, n, k, _rows(h, y, n, "y"), _stream(stream)))


def ep_expert_gemm_swiglu(h: EpHandle, x: torch.Tensor, w: torch.Tensor, act: torch.Tensor,
                          pre: Optional[torch.Tensor] = None, stream=None):
    """act[r] = silu(gate) * up of w[e] x[r]; w [E, 2*ffn, in], gate rows
    first.  pre, when given, keeps the unactivated [R, 2*ffn]."""
    wp, n, k = _expert_weights(h, w, "w")
    f = _gated(n, "w")
    _check(_lib.ep_expert_gemm_swiglu(h.c, _rows(h, x, k, "x"), wp, f, k,
                                      None if pre is None else _rows(h, pre, n, "pre"),
                                      _rows(h, act, f, "act"), _stream(stream)))


def ep_expert_dgrad(h: EpHandle, dy: torch.Tensor, w: torch.Tensor, dx: torch.Tensor, stream=None):
    """dx[r] = transpose(w[e]) dy[r]."""
    wp, n, k = _expert_weights(h, w, "w")
    _check(_lib.ep_expert_dgrad(h.c, _rows(h, dy, n, "dy"), wp, n, k, _rows(h, dx, k, "dx"), _stream(stream)))


def ep_expert_dgrad_swiglu(h: EpHandle, dy: torch.Tensor, w: torch.Tensor, pre: torch.Tensor,
                           dpre: torch.Tensor, stream=None):
    """transpose(w[e]) dy[r] taken through the gated activation; pre and
    dpre [R, 2*ffn], w [E, out, ffn]."""
    wp, n, f = _expert_weights(h, w, "w")
    _check(_lib.ep_expert_dgrad_swiglu(h.c, _rows(h, dy, n, "dy"), wp, _rows(h, pre, 2 * f, "pre"), n, f,
                                       _rows(h, dpre, 2 * f, "dpre"), _stream(stream)))


def ep_expert_wgrad(h: EpHandle, dy: torch.Tensor, x: torch.Tensor, dw: torch.Tensor,
                    accumulate: bool = False, stream=None):
    """dw[e] = (dw[e] +) sum over the expert's rows of dy[r] x[r]^T; dw
    [E, out, in] of the payload type or float32."""
    if dw.dtype not in (torch.float32, _payload(h)):
        raise TypeError("dw must be float32 or %s, got %s" % (_payload(h), dw.dtype))
    wp, n, k = _expert_weights(h, dw, "dw", dw.dtype)
    code = DTYPE_CODES["fp32"] if dw.dtype == torch.float32 else _dtype_code(dw.dtype)
    _check(_lib.ep_expert_wgrad(h.c, _rows(h, dy, n, "dy"), _rows(h, x, k, "x"), n, k, wp, code,
                                1 if accumulate else 0, _stream(stream)))


def _w4(h: EpHandle, wq: torch.Tensor, scales: torch.Tensor):
    wp, n, half = _expert_weights(h, wq, "wq", torch.uint8)
    sp, sn, groups = _expert_weights(h, scales, "scales")
    if sn != n or groups < 1 or (2 * half) % groups:
        raise ValueError("scales must be [%d, %d, in/group], got %s" % (wq.shape[0], n, tuple(scales.shape)))
    return wp, sp, n, 2 * half, 2 * half // groups


def ep_expert_gemv_w4(h: EpHandle, x: torch.Tensor, wq: torch.Tensor, scales: torch.Tensor,
                      y: torch.Tensor, stream=None):
    """y[r] = w[e] x[r] with 4-bit weights: wq uint8 [E, out, in/2] (see
    pack_w4), scales [E, out, in/group] of the payload type.  For up to some
    32 rows per expert; with more, ep_expert_gemm on 16-bit weights is faster."""
    wp, sp, n, k, group = _w4(h, wq, scales)
    _check(_lib.ep_expert_gemv_w4(h.c, _rows(h, x, k, "x"), wp, sp, n, k, group, _rows(h, y, n, "y"),
                                  _stream(stream)))


def ep_expert_gemv_w4_swiglu(h: EpHandle, x: torch.Tensor, wq: torch.Tensor, scales: torch.Tensor,
                             act: torch.Tensor, stream=None):
    """act[r] = silu(gate) * up with 4-bit weights: wq [E, 2*ffn, in/2]."""
    wp, sp, n, k, group = _w4(h, wq, scales)
    f = _gated(n, "wq")
    _check(_lib.ep_expert_gemv_w4_swiglu(h.c, _rows(h, x, k, "x"), wp, sp, f, k, group,
                                         _rows(h, act, f, "act"), _stream(stream)))


def pack_w4(w: torch.Tensor, group: int):
    """Round weights [E, out, in] to 4 bits with one scale per `group` of the
    input features: (wq uint8 [E, out, in/2], scales [E, out, in/group] of
    w's type).  Laid out once, when weights are loaded; plain torch."""
    E, n, k = w.shape
    if group < 1 or k % group or k % 2:
        raise ValueError("in_features %d must be even and a multiple of the group %d" % (k, group))
    g = w.float().view(E, n, k // group, group)
    scales = (g.abs().amax(dim=3) / 7).to(w.dtype)
    s = scales.float().unsqueeze(3)
    q = torch.where(s > 0, torch.round(g / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(g))
    q = (q.clamp(-8, 7) + 8).to(torch.uint8).view(E, n, k)
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous(), scales.contiguous()


# ----------------------------------------------------------------------------
# Router
# ----------------------------------------------------------------------------

_router_configs = {}  # arguments -> RouterConfig


def _router_config(logits, top_k, num_groups, topk_groups, score, normalize, scale) -> RouterConfig:
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens, experts], got %s" % (tuple(logits.shape),))
    key = (logits.shape[1], top_k, num_groups, topk_groups, score, bool(normalize), logits.dtype, scale)
    cfg = _router_configs.get(key)
    if cfg is None:
        if score not in SCORE_CODES:
            raise ValueError("score must be softmax or sigmoid, got %s" % score)
        cfg = RouterConfig(logits.shape[1], top_k, num_groups, topk_groups, SCORE_CODES[score],
                           1 if normalize else 0, _dtype_code(logits.dtype), scale)
        if len(_router_configs) < 1024:
            _router_configs[key] = cfg
    return cfg


def _routes(t: torch.Tensor, T: int, K: int, name: str):
    if t.dim() != 2 or t.shape[0] != T or t.shape[1] != K:
        raise ValueError("%s must be [%d, %d], got %s" % (name, T, K, tuple(t.shape)))


def ep_router(logits: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
              bias: Optional[torch.Tensor] = None, score: str = "softmax", normalize: bool = True,
              num_groups: int = 1, topk_groups: int = 1, scale: float = 1.0, stream=None):
    """The chosen experts and their weights, from logits [T, E]: topk_idx
    int64 [T, K] and topk_weights float32 [T, K] as ep_prepare and
    ep_dispatch take them.  Groups are ranked by the sum of their two largest
    selection values: with the softmax score those are logits, not
    probabilities."""
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [tokens, top_k], got %s" % (tuple(topk_idx.shape),))
    cfg = _router_config(logits, topk_idx.shape[1], num_groups, topk_groups, score, normalize, scale)
    T, K = logits.shape[0], topk_idx.shape[1]
    _routes(topk_idx, T, K, "topk_idx")
    _routes(topk_weights, T, K, "topk_weights")
    if bias is not None and tuple(bias.shape) != (logits.shape[1],):
        raise ValueError("bias must be [%d], got %s" % (logits.shape[1], tuple(bias.shape)))
    _check(_lib.ep_router(cfg, _ptr(logits, None, "logits"), _ptr(bias, torch.float32, "bias"), T,
                          _ptr(topk_idx, torch.int64, "topk_idx"),
                          _ptr(topk_weights, torch.float32, "topk_weights"), _stream(stream)))


def ep_router_bwd(logits: torch.Tensor, topk_idx: torch.Tensor, grad_topk_weights: torch.Tensor,
                  grad_logits: torch.Tensor, score: str = "softmax", normalize: bool = True,
                  scale: float = 1.0, stream=None):
    """grad_logits [T, E] (every element written) from the weights' gradient
    (ep_dispatch_bwd's grad_topk_weights), the choice held fixed."""
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [tokens, top_k], got %s" % (tuple(topk_idx.shape),))
    cfg = _router_config(logits, topk_idx.shape[1], 1, 1, score, normalize, scale)
    T, K = logits.shape[0], topk_idx.shape[1]
    _routes(topk_idx, T, K, "topk_idx")
    _routes(grad_topk_weights, T, K, "grad_topk_weights")
    if grad_logits.shape != logits.shape:
        raise ValueError("grad_logits must be %s, got %s" % (tuple(logits.shape), tuple(grad_logits.shape)))
    _check(_lib.ep_router_bwd(cfg, _ptr(logits, None, "logits"), _ptr(topk_idx, torch.int64, "topk_idx"),
                              _ptr(grad_topk_weights, torch.float32, "grad_topk_weights"), T,
                              _ptr(grad_logits, logits.dtype, "grad_logits"), _stream(stream)))
