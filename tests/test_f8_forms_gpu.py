"""8-bit products and quantisation on handles of other forms than
test_f8_products_gpu.py's: a sharded layer's own experts, alignments of 128 and
more, and experts whose rows fill several row blocks in every product.  The
checks and their tolerances are that module's.
"""
import pytest
import torch

from combine_ep_prepare_gb300 import workloads as wl
from tests import test_f8_products_gpu as products
from tests import test_f8_rows_gpu as quantising
from tests.test_experts_gpu import Step, ep  # noqa: F401

pytestmark = pytest.mark.gpu


class OwnerStep(Step):
    """Rank `rank` of two: E of 2 E experts are its own."""
    rank = 0

    def __init__(self, ep, E, K, T, A, dtype, seed, p_mask=0.1):  # noqa: F811
        self.E, self.dtype, self.tt = E, dtype, wl.TORCH_PAYLOAD[dtype]
        ranks, local, handles = 2, [], []
        for r in range(ranks):
            idx = wl.random_routing(T, K, ranks * E, seed + r, p_mask=p_mask)[0].cuda()
            lid, size = ep.ep_register_layer_sharded(ranks * E, K, 64, T, ranks, r, A, dtype=dtype)
            handles.append((ep.alloc_handle(lid, size), ep.ep_recv_capacity(lid), idx))
            local.append(torch.empty(ranks * E, dtype=torch.int32, device="cuda"))
            ep.ep_shard_count(handles[r][0], idx, local[r])
        self.h, self.R, idx = handles[self.rank]
        counts, off = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
        ep.ep_shard_prepare(self.h, idx, torch.stack(local), counts, A)
        ep.ep_expert_offsets(self.h, off)
        self.counts, self.off = counts.tolist(), off.tolist()
        self.P = self.off[-1]
        self.spans = [(e, slice(self.off[e], self.off[e] + self.counts[e])) for e in range(E) if self.counts[e]]
        self.live = torch.zeros(self.R, dtype=torch.bool)
        for _, r in self.spans:
            self.live[r] = True
        self.pad = ~self.live
        self.pad[self.P:] = False


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("A", [1, 16])
@pytest.mark.parametrize("rank", [0, 1])
def test_sharded_owner(ep, monkeypatch, rank, A, dtype):  # noqa: F811
    monkeypatch.setattr(OwnerStep, "rank", rank)
    for module in (products, quantising):
        monkeypatch.setattr(module, "Step", OwnerStep)
    for shape in ((4, 2, 100, 144, 272), (2, 1, 600, 256, 128)):
        products.test_gemm(ep, shape, A, dtype)
        products.test_dgrad(ep, shape, A, dtype)
    for shape in ((4, 2, 100, 144, 256), (2, 1, 600, 272, 128)):
        products.test_gemm_swiglu(ep, shape, A, dtype)
        products.test_dgrad_swiglu(ep, shape, A, dtype)
    quantising.test_expert_quantize_leaves_other_rows(ep, 4, 2, 100, 528, A, 0.1)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("A", [128, 300])
@pytest.mark.parametrize("E,K,T", [(1, 1, 1), (16, 2, 9), (8, 2, 500), (3, 1, 1000)])
def test_wide_alignments(ep, E, K, T, A, dtype):  # noqa: F811
    """Padding of more than a tile's rows, and experts without a row among others."""
    products.test_gemm(ep, (E, K, T, 272, 400), A, dtype)
    products.test_dgrad(ep, (E, K, T, 272, 400), A, dtype)
    products.test_gemm_swiglu(ep, (E, K, T, 144, 256), A, dtype)
    products.test_dgrad_swiglu(ep, (E, K, T, 144, 256), A, dtype)
    quantising.test_expert_quantize_leaves_other_rows(ep, E, K, T, 400, A, 0.1)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("A", [1, 16])
@pytest.mark.parametrize("shape", [(1, 1, 257, 128, 128), (1, 1, 1300, 272, 384), (2, 1, 1300, 2048, 256), (3, 2, 1100, 16, 1152)], ids=str)
def test_several_row_blocks_in_every_product(ep, shape, A, dtype):  # noqa: F811
    E, K, T, n, f = shape
    products.test_gemm(ep, shape, A, dtype)
    products.test_dgrad(ep, shape, A, dtype)
    products.test_gemm_swiglu(ep, shape, A, dtype)
    products.test_dgrad_swiglu(ep, shape, A, dtype)
