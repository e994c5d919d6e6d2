"""Products of 16-bit rows over long reductions.

Tolerances.  Element by element, those of test_experts_gpu.py.  On norms: the
tensor core truncates as it adds, 1.2e-9 of the norm for each element of a sum
of random terms, and a sum is taken in parts of 32,768 elements, 4e-5; 6e-5 is
allowed beyond what rounding the 64-bit result alone leaves, and 2e-4 behind
the activation (whose slope is at most three here).
A float32 weight gradient is summed in runs of 768 rows, each added in float32
with rounding to nearest.  A run's truncating accumulations leave 1e-6 (768
rows at 1.3e-9); the additions 2^-25 each, as a random walk whose steps are of the
size of the sum so far: 2^-25 * sqrt(n / 2) of the norm for n of them.
"""
import pytest
import torch

from tests.test_experts_gpu import STEP, TINY, UNIT, Step, ep, product  # noqa: F401

pytestmark = pytest.mark.gpu

PART, BEHIND_ACTIVATION = 6e-5, 2e-4


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def check_norm(got, want, extra):
    assert off(got, want) <= off(want.to(got.dtype), want) + extra, (off(got, want), off(want.to(got.dtype), want))


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_weight_gradients_of_long_and_short_experts(ep, dtype, accumulate):  # noqa: F811
    """Several tiles to each pair of SMs, whole sums and sums in parts in turn."""
    counts, n_in, n_out = [40000, 3, 0, 33000, 100, 70000, 32768, 32769], 1032, 1544
    idx = torch.repeat_interleave(torch.arange(8), torch.tensor(counts)).view(-1, 1)
    s = Step(ep, 8, 1, idx.shape[0], 1, dtype, 31, idx=idx)
    assert s.counts == counts
    g = torch.Generator(device="cuda").manual_seed(32)
    dy = (torch.randn(s.R, n_out, generator=g, device="cuda") * 2.0 ** -6).to(s.tt)
    x = torch.randn(s.R, n_in, generator=g, device="cuda").to(s.tt)
    dw = torch.randn(8, n_out, n_in, generator=g, device="cuda").to(s.tt)
    before = dw.clone()
    ep.ep_expert_wgrad(s.h, dy, x, dw, accumulate=accumulate)
    for e in range(8):
        r = slice(s.off[e], s.off[e] + counts[e])
        want, mag = product(dy[r].t(), x[r])
        bound = counts[e] * STEP * mag
        if accumulate:
            want = want + before[e].double()
        bound = bound + (UNIT[dtype] + 2.0 ** -24) * (want.abs() + bound) + TINY[dtype]
        assert bool(((dw[e].double() - want).abs() <= bound).all()), e
        if counts[e]:
            check_norm(dw[e], want, PART)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [200000, 1 << 20])
def test_one_long_expert(ep, dtype, rows):  # noqa: F811
    s = Step(ep, 1, 1, rows, 1, dtype, 33, idx=torch.zeros(rows, 1, dtype=torch.int64))
    g = torch.Generator(device="cuda").manual_seed(34)
    dy = torch.randn(rows, 72, generator=g, device="cuda").to(s.tt)
    x = torch.randn(rows, 136, generator=g, device="cuda").to(s.tt)
    dw = torch.empty(1, 72, 136, dtype=s.tt, device="cuda")
    ep.ep_expert_wgrad(s.h, dy, x, dw)
    check_norm(dw[0], dy.double().t() @ x.double(), PART)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("E,T,n_in,n_out", [(4, 2400, 33032, 4096), (1, 1, 1 << 20, 8), (2, 40, 262144, 72), (3, 300, 32768, 136)])
def test_forward_of_many_features(ep, dtype, E, T, n_in, n_out):  # noqa: F811
    idx = (torch.arange(T) % E).view(-1, 1)
    s = Step(ep, E, 1, T, 1, dtype, 35, idx=idx)
    g = torch.Generator(device="cuda").manual_seed(36)
    x = torch.randn(s.R, n_in, generator=g, device="cuda").to(s.tt)
    w = (torch.randn(E, n_out, n_in, generator=g, device="cuda") * n_in ** -0.5).to(s.tt)
    y = s.out(n_out)
    ep.ep_expert_gemm(s.h, x, w, y)
    want, mag = s.per_row(lambda e, r: product(x[r], w[e].t()), n_out)
    s.check_rows(y, want, n_in * STEP * mag + UNIT[dtype] * want.abs())
    check_norm(y, want, PART if T > 1 else 2 * PART)  # eight values: no average


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gated_forward_and_input_gradients_of_many_features(ep, dtype):  # noqa: F811
    E, T, wide, f = 2, 90, 98312, 136
    s = Step(ep, E, 1, T, 8, dtype, 37, idx=(torch.arange(T) % E).view(-1, 1))
    live = s.live.cuda()
    x, w = s.rows(wide, 38), s.weights(2 * f, wide, 39)
    act, pre = s.out(f), s.out(2 * f)
    ep.ep_expert_gemm_swiglu(s.h, x, w, act, pre=pre)
    want, _ = s.per_row(lambda e, r: product(x[r], w[e].t()), 2 * f)
    check_norm(pre[live], want[live], PART)
    check_norm(act[live], (torch.nn.functional.silu(want[:, :f]) * want[:, f:])[live], BEHIND_ACTIVATION)
    dy = x
    w2 = (s.weights(wide, f, 40).float() * (f / wide) ** 0.5).to(s.tt)  # the sum runs over its rows
    da, dpre = s.out(f), s.out(2 * f)
    ep.ep_expert_dgrad(s.h, dy, w2, da)
    ep.ep_expert_dgrad_swiglu(s.h, dy, w2, pre, dpre)
    want, _ = s.per_row(lambda e, r: product(dy[r], w2[e]), f)
    check_norm(da[live], want[live], PART)
    p = torch.nan_to_num(pre.double()).requires_grad_()
    wanted = torch.autograd.grad(torch.nn.functional.silu(p[:, :f]) * p[:, f:], p, want)[0]
    check_norm(dpre[live], wanted[live], BEHIND_ACTIVATION)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [768, 2000, 20000, 200000, 1 << 22])
def test_float32_gradients_of_16_bit_rows(ep, rows, dtype, accumulate):  # noqa: F811
    """What the header promises: 1.4e-6 of the norm up to 200,000 rows, 2.6e-6 at four million."""
    s = Step(ep, 1, 1, rows, 1, dtype, 41, idx=torch.zeros(rows, 1, dtype=torch.int64))
    g = torch.Generator(device="cuda").manual_seed(42)
    dy = torch.randn(rows, 72, generator=g, device="cuda").to(s.tt)
    x = torch.randn(rows, 136, generator=g, device="cuda").to(s.tt)
    dw = torch.randn(1, 72, 136, generator=g, device="cuda")
    want = dw[0].double() if accumulate else 0
    for i in range(0, rows, 1 << 16):
        want = want + dy[i:i + (1 << 16)].double().t() @ x[i:i + (1 << 16)].double()
    ep.ep_expert_wgrad(s.h, dy, x, dw, accumulate=accumulate)
    bound = 1e-6 + 2.0 ** -25 * (rows / 768 / 2) ** 0.5
    assert bound <= (1.4e-6 if rows <= 200000 else 2.6e-6)
    assert off(dw[0], want) <= bound
