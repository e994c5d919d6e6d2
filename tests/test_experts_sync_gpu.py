"""Expert products where one part of a kernel hands data to another: the 4-bit
scales that a warp's lanes share stage by stage.

Tolerances are those of test_experts_gpu.py: n * 2^-23 of the sum of the terms'
magnitudes, then one rounding to the output type.
"""
import pytest
import torch

from tests.test_experts_gpu import STEP, UNIT, Step, ep, product, w4_weights  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1, 1, 2048, 64), (8, 4, 40, 1152, 136), (64, 8, 64, 2048, 264)], ids=str)
def test_scales_of_one_stage_never_meet_another_stage(ep, shape, group, dtype):  # noqa: F811
    """Scales of neighbouring stages (256 reduction elements) differ by 2^6, so
    a scale taken a stage too early or too late is far outside the bound."""
    E, K, T, n_in, n_out = shape
    s = Step(ep, E, K, T, 1, dtype, 14, p_mask=0.0)
    x = s.rows(n_in, 91)
    wq, sc, _ = w4_weights(s, n_out, n_in, group, 92)
    stage = torch.arange(n_in // group, device="cuda") * group // 256
    sc = sc * torch.where(stage % 2 == 0, 1.0, 2.0 ** -6).to(sc.dtype)
    q = torch.stack([wq & 15, wq >> 4], dim=3).flatten(2).double() - 8
    w = q * sc.double().repeat_interleave(group, dim=2)
    for _ in range(8):
        y = s.out(n_out)
        ep.ep_expert_gemv_w4(s.h, x, wq, sc, y)
        want, mag = s.per_row(lambda e, r: product(x[r], w[e].t()), n_out)
        s.check_rows(y, want, (n_in + 2) * STEP * mag + UNIT[dtype] * want.abs())
