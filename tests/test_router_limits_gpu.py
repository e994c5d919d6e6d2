"""Router scores and gradients at the ends of their range.

Tolerances.  A sigmoid and its complement are each good to a few units in the
last place however close to 0 or 1, sums of K terms and the products around
them add K + 16 rounding errors of 2^-23, relative to the sum of the
magnitudes of a gradient's terms, its factor 1 - s among them; then one
rounding to the logits' type.
"""
import pytest
import torch

from tests.test_router_gpu import TYPES, UNIT, ep  # noqa: F401

pytestmark = pytest.mark.gpu

TINY = {"fp32": 2.0 ** -120, "bf16": 2.0 ** -120, "fp16": 2.0 ** -24}


def gradient(ep, z, idx, g, **kw):
    gz = torch.full(z.shape, float("nan"), dtype=z.dtype, device="cuda")
    ep.ep_router_bwd(z, idx, g, gz, score="sigmoid", **kw)
    return gz.double().gather(1, idx)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("low,high,size", [(8, 20, 1.0), (14, 60, 1.0), (-20, -8, 1.0), (-87, -84, 64.0), (-20, 20, 1.0)])
def test_sigmoid_gradient_of_confident_logits(ep, low, high, size, normalize, dtype):  # noqa: F811
    T, E, K = 200, 24, 4
    gen = torch.Generator().manual_seed(21)
    z = (low + (high - low) * torch.rand(T, E, generator=gen)).to(TYPES[dtype]).cuda()
    idx = torch.rand(T, E, generator=gen).argsort(1)[:, :K].contiguous().cuda()
    g = (torch.randn(T, K, generator=gen) * size).cuda()
    got = gradient(ep, z, idx, g, normalize=normalize, scale=0.7)
    zk, g = z.double().gather(1, idx), g.double() * 0.7
    s, rest = torch.sigmoid(zk), torch.sigmoid(-zk)
    w = s / s.sum(1, keepdim=True) if normalize else s
    if normalize:
        want = w * rest * (g - (g * w).sum(1, keepdim=True))
        size = w * rest * (g.abs() + (g.abs() * w).sum(1, keepdim=True))
    else:
        want = w * rest * g
        size = want.abs()
    bound = (K + 16) * 2.0 ** -23 * size + UNIT[dtype] * want.abs() + TINY[dtype]
    d = (got - want).abs()
    assert bool((d <= bound).all()), (d / bound).max().item()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("normalize", [True, False])
def test_an_infinite_logit_shows_in_its_row_alone(ep, normalize, dtype):  # noqa: F811
    """exp(inf - inf): the softmax of a row with +infinity is NaN, not a set of
    zero weights that would drop the token unseen."""
    T, E, K = 9, 40, 5
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(22)).to(TYPES[dtype])
    z[4, 17] = float("inf")
    z = z.cuda()
    idx, w = torch.empty(T, K, dtype=torch.int64, device="cuda"), torch.empty(T, K, device="cuda")
    ep.ep_router(z, idx, w, normalize=normalize)
    assert idx[4, 0].item() == 17 and bool((idx >= 0).all())
    gz = torch.zeros_like(z)
    ep.ep_router_bwd(z, idx, torch.ones_like(w), gz, normalize=normalize)
    row = torch.arange(T, device="cuda") == 4
    assert bool(torch.isnan(w[row]).all()) and bool(torch.isfinite(w[~row]).all())
    assert bool(torch.isnan(gz.gather(1, idx)[row]).all()) and bool(torch.isfinite(gz[~row]).all())
