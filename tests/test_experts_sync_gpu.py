"""Expert products where one part of a kernel hands data to another: the 4-bit
scales that a warp's lanes share stage by stage, and the rows past an expert's
last that are zeroed before the weight gradient's tensor-core products.

Tolerances are those of test_experts_gpu.py: n * 2^-23 of the sum of the terms'
magnitudes, then one rounding to the output type.
"""
import pytest
import torch

from tests.test_experts_gpu import STEP, TINY, UNIT, Step, ep, product, w4_weights  # noqa: F401

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


@pytest.mark.parametrize("wtype", ["payload", "fp32"])
@pytest.mark.parametrize("A", [1, 16])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_weight_gradients_of_every_row_count_leave_out_the_rows_behind(ep, dtype, A, wtype):  # noqa: F811
    """Experts of 1 to 130 rows, features for both blocks of a pair and for
    ragged tiles.  What lies behind an expert's rows is NaN (A = 16) or the
    next expert's rows, 2^6 times larger (A = 1)."""
    E, n_in, n_out = 130, 264, 392
    idx = torch.repeat_interleave(torch.arange(E), torch.arange(1, E + 1)).view(-1, 1)
    s = Step(ep, E, 1, idx.shape[0], A, dtype, 15, idx=idx)
    assert s.counts == list(range(1, E + 1))
    dy, x = s.rows(n_out, 93), s.rows(n_in, 94)
    if A == 1:
        for e, r in s.spans:
            dy[r] *= 2.0 ** (6 * (e % 2))
            x[r] *= 2.0 ** (6 * (e % 2))
    tt = torch.float32 if wtype == "fp32" else s.tt
    first = None
    for _ in range(4):
        dw = torch.full((E, n_out, n_in), float("nan"), dtype=tt, device="cuda")
        ep.ep_expert_wgrad(s.h, dy, x, dw)
        first = dw if first is None else first
        assert torch.equal(dw, first)
    for e, r in s.spans:
        want, mag = product(dy[r].t(), x[r])
        unit = UNIT["fp32" if wtype == "fp32" else dtype]
        bound = s.counts[e] * STEP * mag + unit * (want.abs() + s.counts[e] * STEP * mag) + TINY["fp32" if wtype == "fp32" else dtype]
        got = first[e].double()
        over = (want.abs() + bound > torch.finfo(tt).max) & (got == torch.inf * want.sign())  # rounded to infinity in fp16
        assert bool((((got - want).abs() <= bound) | over).all()), e
