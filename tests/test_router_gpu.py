"""Router and its gradient against the definition.

The choice is compared exactly: with a Python restatement in float32 selection
values where the values are logits or logits-derived ties, and in float64 with
near-ties excluded where they go through a sigmoid.  Weights: a float32
exponential is good to 2 units in the last place, a sum of n terms and two
divisions add n + 4 rounding errors: (n + 8) * 2^-23 relative.  Gradients: the
same relative to the sum of the magnitudes of their terms, plus one rounding
to the logits' type.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_ep_prepare_gb300 as ep
    return ep


def choose(z, bias, K, groups, kept, sigmoid):
    """The definition, row by row: z float64 numpy [T, E]; returns ids and how
    far the closest rejected alternative was."""
    T, E = z.shape
    per = E // groups
    with np.errstate(over="ignore", invalid="ignore"):
        v = 1 / (1 + np.exp(-z)) + (0 if bias is None else bias) if sigmoid else z.copy()
    v[~(z > -np.inf) | ~(v > -np.inf)] = -np.inf
    ids = np.full((T, K), -1, dtype=np.int64)
    gap = np.full(T, np.inf)
    for t in range(T):
        row = v[t].copy()
        if groups > 1:
            rank = []
            for g in range(groups):
                a = np.sort(row[g * per:(g + 1) * per])[::-1]
                best = a[0]
                second = a[1] if per > 1 and a[1] > -np.inf else best
                rank.append(best + second if best > -np.inf else -np.inf)
            rank = np.array(rank)
            order = np.argsort(-rank, kind="stable")
            if kept < groups and rank[order[kept]] > -np.inf:
                gap[t] = min(gap[t], rank[order[kept - 1]] - rank[order[kept]])
            for g in order[kept:]:
                row[g * per:(g + 1) * per] = -np.inf
        order = np.argsort(-row, kind="stable")
        take = [e for e in order[:K] if row[e] > -np.inf]
        ids[t, :len(take)] = take
        vals = row[order[:K + 1]]
        vals = vals[vals > -np.inf]
        if len(vals) > 1:
            gap[t] = min(gap[t], np.min(vals[:-1] - vals[1:]))
    return ids, gap


def weights(z, ids, sigmoid, normalize, scale):
    T, E = z.shape
    ok = ids >= 0
    zs = np.where(ok, np.take_along_axis(z, np.maximum(ids, 0), 1), -np.inf)
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            s = np.where(ok, 1 / (1 + np.exp(-zs)), 0)
        else:
            can = np.where(z > -np.inf, z, -np.inf)
            m = can.max(1, keepdims=True)
            m = np.where(m > -np.inf, m, 0)
            s = np.where(ok, np.exp(zs - m), 0)
            if not normalize:
                s = s / np.maximum(np.exp(can - m).sum(1, keepdims=True), 1e-300)
        if normalize:
            tot = s.sum(1, keepdims=True)
            s = np.where(tot > 0, s / np.where(tot > 0, tot, 1), 0)
    return s * scale


# T, E, K, groups, kept
SHAPES = [(1, 1, 1, 1, 1), (3, 5, 5, 1, 1), (17, 33, 7, 1, 1), (200, 64, 6, 8, 3), (300, 256, 8, 8, 4), (65, 1024, 32, 32, 5),
          (40, 96, 4, 32, 1), (128, 1000, 9, 4, 2), (50, 16, 4, 16, 7)]


def make(T, E, dtype, seed, ties=False, holes=False):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * 2
    if ties:
        z = torch.randint(-2, 3, (T, E), generator=g).float()
    if holes:
        z[torch.rand(T, E, generator=g) < 0.4] = -float("inf")
        z[torch.rand(T, E, generator=g) < 0.1] = float("nan")
        z[torch.rand(T, E, generator=g) < 0.1] = torch.finfo(TYPES[dtype]).min
        z[T // 2] = -float("inf")
    return z.to(TYPES[dtype])


def call(ep, z, K, **kw):
    idx = torch.full((z.shape[0], K), -7, dtype=torch.int64, device="cuda")
    w = torch.full((z.shape[0], K), float("nan"), device="cuda")
    ep.ep_router(z.cuda(), idx, w, **kw)
    return idx.cpu().numpy(), w.cpu().double().numpy()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("kind", ["plain", "ties", "holes"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_softmax(ep, shape, kind, normalize, dtype):
    T, E, K, groups, kept = shape
    z = make(T, E, dtype, 1, ties=kind == "ties", holes=kind == "holes")
    idx, w = call(ep, z, K, score="softmax", normalize=normalize, num_groups=groups, topk_groups=kept, scale=1.5)
    z64 = z.double().numpy()
    # group ranks are float32 sums of two logits
    want, gap = choose(z64, None, K, groups, kept, False)
    sure = (gap > 1e-5) | (gap == 0) if groups > 1 and kind != "ties" else np.ones(T, bool)
    assert sure.mean() > 0.9
    assert np.array_equal(idx[sure], want[sure])
    ww = weights(z64, idx, False, normalize, 1.5)
    assert np.all(np.abs(w - ww) <= (E + 8) * 2.0 ** -23 * ww + 2.0 ** -125)


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("holes", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_sigmoid(ep, shape, holes, normalize, bias):
    T, E, K, groups, kept = shape
    z = make(T, E, "fp32", 2, holes=holes)
    if holes:  # two saturated logits of a row would be near-ties of sigmoid 0
        z[z == torch.finfo(torch.float32).min] = -float("inf")
    b = torch.randn(E, generator=torch.Generator().manual_seed(3)) * 0.2 if bias else None
    idx, w = call(ep, z, K, score="sigmoid", normalize=normalize, num_groups=groups, topk_groups=kept,
                  bias=None if b is None else b.cuda())
    z64 = z.double().numpy()
    want, gap = choose(z64, None if b is None else b.double().numpy(), K, groups, kept, True)
    sure = gap > 2e-6
    assert sure.mean() > 0.8
    assert np.array_equal(idx[sure], want[sure])
    ww = weights(z64, idx, True, normalize, 1.0)
    assert np.all(np.abs(w - ww) <= (K + 8) * 2.0 ** -23 * ww + 2.0 ** -125)


def test_sigmoid_matches_the_elementary_form_bit_for_bit(ep):
    """1 / (1 + exp(-z)) + b in float32, sorted stably: the ids agree exactly."""
    T, E, K = 4096, 256, 8
    z = make(T, E, "fp32", 4).cuda()
    b = (torch.randn(E, generator=torch.Generator().manual_seed(5)) * 0.1).cuda()
    v = 1 / (1 + torch.exp(-z)) + b
    want = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :K]
    idx, _ = call(ep, z, K, score="sigmoid", bias=b)
    assert np.array_equal(idx, want.cpu().numpy())


def test_bias_that_masks(ep):
    z = make(30, 16, "fp32", 6)
    b = torch.zeros(16)
    b[3:] = -float("inf")
    idx, w = call(ep, z, 4, score="sigmoid", bias=b.cuda())
    assert np.array_equal(np.sort(idx, 1), np.tile([-1, 0, 1, 2], (30, 1)))
    assert np.all(w[:, 3] == 0) and np.allclose(w.sum(1), 1)


def test_no_tokens(ep):
    ep.ep_router(torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int64, device="cuda"),
                 torch.empty(0, 2, device="cuda"))
    ep.ep_router_bwd(torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int64, device="cuda"),
                     torch.empty(0, 2, device="cuda"), torch.empty(0, 8, device="cuda"))


def reference_grad(z, idx, g, sigmoid, normalize, scale):
    """Autograd in float64 over the rows' choosable logits; also the sum of
    the magnitudes of the gradient's terms."""
    z64 = z.double()
    can = z64 > -float("inf")
    zz = torch.where(can, z64, torch.full_like(z64, -1e300)).requires_grad_()
    ok = idx >= 0
    at = idx.clamp_min(0)
    if sigmoid:
        s = torch.sigmoid(zz).gather(1, at) * ok
        w = s / s.sum(1, keepdim=True).clamp_min(1e-300) if normalize else s
    elif normalize:
        w = torch.softmax(torch.where(ok, zz.gather(1, at), torch.full_like(g.double(), -1e300)), 1) * ok
    else:
        w = torch.softmax(zz, 1).gather(1, at) * ok
    gg = g.double() * scale
    grad = torch.autograd.grad((w * gg).sum(), zz)[0]
    term = (w.detach() * gg.abs()).sum(1, keepdim=True)
    spread = torch.zeros_like(z64).scatter_add(1, at, w.detach() * gg.abs() * ok)
    if not sigmoid and not normalize:
        base = torch.softmax(zz.detach(), 1)
        return grad, base * term + spread
    chosen = torch.zeros_like(z64).scatter_add(1, at, w.detach() * ok)
    return grad, chosen * term + spread


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("holes", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradient(ep, shape, holes, normalize, score, dtype):
    T, E, K, groups, kept = shape
    z = make(T, E, dtype, 7, holes=holes).cuda()
    idx = torch.empty(T, K, dtype=torch.int64, device="cuda")
    w = torch.empty(T, K, device="cuda")
    ep.ep_router(z, idx, w, score=score, normalize=normalize, num_groups=groups, topk_groups=kept, scale=0.7)
    g = torch.randn(T, K, generator=torch.Generator().manual_seed(8)).cuda()
    gz = torch.full((T, E), float("nan"), dtype=z.dtype, device="cuda")
    ep.ep_router_bwd(z, idx, g, gz, score=score, normalize=normalize, scale=0.7)
    want, mag = reference_grad(z, idx, g, score == "sigmoid", normalize, 0.7)
    d = (gz.double() - want).abs()
    tiny = 2.0 ** -24 if dtype == "fp16" else 2.0 ** -120  # fp16 rounds small gradients to its subnormals
    bound = (E + 16) * 2.0 ** -23 * mag + UNIT[dtype] * want.abs() + tiny
    assert bool((d <= bound).all()), (d / bound).max().item()
    dense = score == "softmax" and not normalize
    if not dense:
        untouched = torch.ones(T, E + 1, dtype=torch.bool, device="cuda")
        untouched.scatter_(1, torch.where(idx >= 0, idx, E), False)
        assert bool((gz[untouched[:, :E]] == 0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(ep, score, normalize):
    """Central differences of sum(w * g) with step 2^-7: the third derivative
    of the scores is below 1, so the difference is off by less than h^2, and
    float32 noise adds 2^-22 / h; choices that the step changes are left out."""
    T, E, K = 64, 24, 4
    z = make(T, E, "fp32", 9).cuda()
    g = torch.randn(T, K, generator=torch.Generator().manual_seed(10)).cuda()
    idx, w = torch.empty(T, K, dtype=torch.int64, device="cuda"), torch.empty(T, K, device="cuda")
    ep.ep_router(z, idx, w, score=score, normalize=normalize)
    gz = torch.empty_like(z)
    ep.ep_router_bwd(z, idx, g, gz, score=score, normalize=normalize)
    d = torch.randn(T, E, generator=torch.Generator().manual_seed(11)).cuda()
    d = d / d.norm(dim=1, keepdim=True)
    h = 2.0 ** -7
    vals, same = [], torch.ones(T, dtype=torch.bool, device="cuda")
    for sign in (1, -1):
        i2, w2 = torch.empty_like(idx), torch.empty_like(w)
        ep.ep_router(z + sign * h * d, i2, w2, score=score, normalize=normalize)
        same &= (i2 == idx).all(1)
        vals.append((w2.double() * g.double()).sum(1))
    diff = (vals[0] - vals[1]) / (2 * h)
    want = (gz.double() * d.double()).sum(1)
    tol = (h * h + 2.0 ** -22 / h) * g.abs().double().sum(1) * 2
    assert same.float().mean() > 0.7
    assert bool(((diff - want).abs()[same] <= tol[same]).all())
