"""The norm's gradient at the largest batch that it takes: 2^31 - 1 rows, past
the last of which a 32-bit signed row number would wrap and be taken for a row.

With h = 1, weight = 1/2, eps = 0 and rows of gradients (2, -2, 2, ...) the
rows' means are 0 and their norms 1, so grad_h is (1, -1, ...) exactly.  A
block's share of grad_weight is 2 * 2^31 / 608 < 2^24, exact in float32; 608 of
them are joined in 608 / 16 + 16 = 54 additions, each off by at most 2^-24.
"""
import pytest
import torch

from tests.test_experts_gpu import ep  # noqa: F401

pytestmark = pytest.mark.gpu


def test_gradient_of_the_most_rows(ep):  # noqa: F811
    T, H = (1 << 31) - 1, 8
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 2.5 * T * H * 2:
        pytest.skip("needs 86 GB of device memory")
    sign = torch.tensor([1.0, -1.0] * (H // 2), dtype=torch.bfloat16, device="cuda")
    dy = (2 * sign).expand(T, H).contiguous()
    h = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    w, dw = torch.full((H,), 0.5, dtype=torch.bfloat16, device="cuda"), torch.empty(H, device="cuda")
    ep.ep_rmsnorm_bwd(dy, h, w, dy, dw, ep.rmsnorm_bwd_workspace(T, H), eps=0.0)  # in place
    assert all(bool((part == sign).all()) for part in dy.split(1 << 27))
    assert bool(((dw.double() - 2.0 * T * sign.double()).abs() <= 54 * 2.0 ** -24 * 2 * T).all())
    del dy, h
    torch.cuda.empty_cache()
