"""Products of 8-bit rows and weights against the same sums in 64 bits.

Tolerances.  Products of e4m3 values are exact in float32.  A block's sum of
at most 128 of them, each addition off by at most 2^-23 (the tensor core may
truncate), is off by 128 * 2^-23 of its magnitudes; multiplying by the two
scales and adding the n / 128 blocks adds (n / 128 + 3) 2^-23.  Then one
rounding to the output type.  The activation passes an error on as in
test_experts_gpu.py; a quantised result lies within half a step of e4m3 (2^-4
of the value, 2^-10 of the scale below) of the exact quotient.
Padding rows and rows past the used ones hold NaN in values and scales.
"""
import pytest
import torch

from combine_ep_prepare_gb300 import workloads as wl
from tests.test_experts_gpu import ACT, STEP, TINY, UNIT, Step, ep  # noqa: F401
from tests.test_f8_rows_gpu import F8, columns, same

pytestmark = pytest.mark.gpu


def sum_bound(n):
    return (128 + (n + 127) // 128 + 3) * STEP


def rows8(ep, s, width, seed):  # noqa: F811
    """Quantised receive rows, NaN wherever no expert owns a row, and their values."""
    x = wl.payload_normal(s.R, width, seed, "fp32") * torch.logspace(-2, 1, (width + 127) // 128).repeat_interleave(128)[:width]
    q, sc = torch.empty(s.R, width, dtype=F8, device="cuda"), torch.empty(s.R, columns(width), device="cuda")
    ep.ep_quantize_rows(x.cuda(), q, sc)
    value = q.double() * sc.double().repeat_interleave(128, 1)[:, :width]
    q.view(torch.uint8)[(~s.live).cuda()] = 0x7f
    sc[(~s.live).cuda()] = float("nan")
    return q, sc, value


def weights8(ep, E, n, k, seed):  # noqa: F811
    w = wl.payload_normal(E * n, k, seed, "fp32").view(E, n, k) * k ** -0.5
    w = w * torch.linspace(0.2, 3, (k + 127) // 128).repeat_interleave(128)[:k] * torch.linspace(3, 0.2, (n + 127) // 128).repeat_interleave(128)[:n, None]
    q, sc = ep.pack_f8(w.cuda())
    return q, sc, q.double() * sc.double().repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]


def per_expert(s, a, w, width):
    want, mag = (torch.zeros(s.R, width, dtype=torch.float64, device="cuda") for _ in range(2))
    for e, r in s.spans:
        want[r], mag[r] = a[r] @ w[e], a[r].abs() @ w[e].abs()
    return want, mag


SHAPES = [(1, 1, 1, 16, 16), (4, 2, 9, 128, 128), (8, 2, 33, 144, 400), (3, 1, 300, 1040, 272), (5, 2, 517, 512, 640),
          (40, 8, 64, 256, 1152), (2, 1, 257, 4096, 256), (130, 1, 1000, 128, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("A", [1, 16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gemm(ep, shape, A, dtype):  # noqa: F811
    E, K, T, n_in, n_out = shape
    s = Step(ep, E, K, T, A, dtype, 30)
    x, xs, xv = rows8(ep, s, n_in, 31)
    w, ws, wv = weights8(ep, E, n_out, n_in, 32)
    y = s.out(n_out)
    ep.ep_expert_gemm_f8(s.h, x, xs, w, ws, y)
    want, mag = per_expert(s, xv, wv.transpose(1, 2), n_out)
    s.check_rows(y, want, sum_bound(n_in) * mag + UNIT[dtype] * (want.abs() + sum_bound(n_in) * mag))
    y2 = s.out(n_out)
    ep.ep_expert_gemm_f8(s.h, x, xs, w, ws, y2)
    assert same(y, y2)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("A", [1, 16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dgrad(ep, shape, A, dtype):  # noqa: F811
    E, K, T, n_in, n_out = shape
    s = Step(ep, E, K, T, A, dtype, 33)
    dy, ds, dv = rows8(ep, s, n_out, 34)
    w, ws, wv = weights8(ep, E, n_out, n_in, 35)
    dx = s.out(n_in)
    ep.ep_expert_dgrad_f8(s.h, dy, ds, w, ws, dx)
    want, mag = per_expert(s, dv, wv, n_in)
    s.check_rows(dx, want, sum_bound(n_out) * mag + UNIT[dtype] * (want.abs() + sum_bound(n_out) * mag))


GATED = [(1, 1, 1, 16, 128), (4, 2, 9, 128, 256), (8, 2, 33, 144, 384), (3, 1, 300, 1040, 128), (40, 8, 64, 256, 640), (2, 1, 513, 2048, 256)]


def act_bounds(pre, mag, f, n):
    g, u = pre[:, :f], pre[:, f:]
    dg, du = sum_bound(n) * mag[:, :f], sum_bound(n) * mag[:, f:]
    sg = torch.sigmoid(g)
    act = g * sg * u
    return act, 1.1 * dg * (u.abs() + du) + (g * sg).abs() * du + ACT * (1 + g.abs()) * act.abs()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("A", [1, 16])
@pytest.mark.parametrize("shape", GATED, ids=str)
def test_gemm_swiglu(ep, shape, A, dtype):  # noqa: F811
    E, K, T, n_in, f = shape
    s = Step(ep, E, K, T, A, dtype, 36)
    x, xs, xv = rows8(ep, s, n_in, 37)
    w, ws, wv = weights8(ep, E, 2 * f, n_in, 38)
    pre, act = s.out(2 * f), s.out(f)
    q = torch.full((s.R, f), 0x35, dtype=torch.uint8, device="cuda")
    qs = torch.full((s.R, columns(f)), 7.0, device="cuda")
    ep.ep_expert_gemm_f8_swiglu(s.h, x, xs, w, ws, act=act, pre=pre, act_q=q.view(F8), act_scales=qs)
    want, mag = per_expert(s, xv, wv.transpose(1, 2), 2 * f)
    s.check_rows(pre, want, sum_bound(n_in) * mag + UNIT[dtype] * (want.abs() + sum_bound(n_in) * mag))
    a, off = act_bounds(want, mag, f, n_in)
    s.check_rows(act, a, off + UNIT[dtype] * (a.abs() + off))
    live = s.live.cuda()
    m = a.abs().view(s.R, -1, 128).amax(2)
    off_m = off.view(s.R, -1, 128).amax(2)
    got = qs[:, :f // 128].double()
    assert bool(((got - m / 448).abs() <= (off_m + 4 * STEP * m) / 448 + 1e-30)[live].all())
    scale = got.repeat_interleave(128, 1)
    value = q.view(F8).double() * scale
    assert bool(((value - a).abs() <= a.abs() * (2.0 ** -4 + 1e-6) + scale * 2.0 ** -10 + 1.1 * off)[live].all())
    pad = s.pad.cuda()
    assert bool((q[pad] == 0).all()) and bool((qs[pad] == 0).all()) and bool((qs[live][:, f // 128:] == 0).all())
    assert bool((q[s.P:] == 0x35).all()) and bool((qs[s.P:] == 7.0).all())
    # each result alone
    for kw in (dict(act=s.out(f)), dict(pre=s.out(2 * f)), dict(act_q=torch.empty_like(q).view(F8), act_scales=torch.empty_like(qs))):
        ep.ep_expert_gemm_f8_swiglu(s.h, x, xs, w, ws, **kw)
        for name, t in kw.items():
            full = {"act": act, "pre": pre, "act_q": q, "act_scales": qs}[name]
            assert same(t[:s.P], full[:s.P]), name


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("A", [1, 16])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16, 128), (8, 2, 33, 144, 384), (3, 1, 300, 1040, 128), (40, 8, 64, 256, 640)], ids=str)
def test_dgrad_swiglu(ep, shape, A, dtype):  # noqa: F811
    E, K, T, n_out, f = shape
    s = Step(ep, E, K, T, A, dtype, 39)
    dy, ds, dv = rows8(ep, s, n_out, 40)
    w, ws, wv = weights8(ep, E, n_out, f, 41)
    pre, dpre = s.rows(2 * f, 42), s.out(2 * f)
    ep.ep_expert_dgrad_f8_swiglu(s.h, dy, ds, w, ws, pre, dpre)
    da, mag = per_expert(s, dv, wv, f)
    g, u = torch.nan_to_num(pre.double()).chunk(2, dim=1)
    sg = torch.sigmoid(g)
    want = torch.cat([da * u * sg * (1 + g * (1 - sg)), da * g * sg], 1)
    slope = torch.cat([(u * sg).abs() * (1 + g.abs()), (g * sg).abs()], 1)
    off = sum_bound(n_out) * mag.repeat(1, 2) * slope + ACT * (1 + g.abs()).repeat(1, 2) * (da.abs().repeat(1, 2) * slope)
    s.check_rows(dpre, want, off + UNIT[dtype] * (want.abs() + off))


def test_forward_and_gradient_are_adjoint(ep):  # noqa: F811
    """sum of y dy over the rows equals sum of x dx: the gradient against the
    forward pass itself (the product is linear in the rows, so a difference
    quotient is exact)."""
    s = Step(ep, 6, 2, 200, 1, "fp16", 43)
    x, xs, xv = rows8(ep, s, 512, 44)
    dy, ds, dv = rows8(ep, s, 384, 45)
    w, ws, wv = weights8(ep, 6, 384, 512, 46)
    y, dx = s.out(384), s.out(512)
    ep.ep_expert_gemm_f8(s.h, x, xs, w, ws, y)
    ep.ep_expert_dgrad_f8(s.h, dy, ds, w, ws, dx)
    live = s.live.cuda()
    a, b = (y.double() * dv)[live].sum(), (dx.double() * xv)[live].sum()
    size = (y.double() * dv)[live].abs().sum() + (dx.double() * xv)[live].abs().sum()
    assert abs(a - b) <= (UNIT["fp16"] + 1e-4) * size


def test_infinite_rows_stay_in_their_row(ep):  # noqa: F811
    s = Step(ep, 2, 1, 40, 1, "bf16", 47, p_mask=0.0)
    x, xs, xv = rows8(ep, s, 256, 48)
    w, ws, wv = weights8(ep, 2, 256, 256, 49)
    y = s.out(256)
    ep.ep_expert_gemm_f8(s.h, x, xs, w, ws, y)
    xs[7, 1] = float("inf")
    x.view(torch.uint8)[9, 130] = 0x7f
    z = s.out(256)
    ep.ep_expert_gemm_f8(s.h, x, xs, w, ws, z)
    assert not bool(torch.isfinite(z[7]).any()) and bool(torch.isnan(z[9]).all())
    keep = torch.ones(s.R, dtype=torch.bool)
    keep[7] = keep[9] = False
    assert same(y[keep.cuda()], z[keep.cuda()])


def test_unprepared_and_empty_batches_write_nothing(ep):  # noqa: F811
    lid, size = ep.ep_register_layer(4, 2, 64, 8)
    R, h = ep.ep_recv_capacity(lid), ep.alloc_handle(lid, size)
    x, xs = torch.zeros(R, 128, dtype=torch.uint8, device="cuda").view(F8), torch.zeros(R, 4, device="cuda")
    w, ws, _ = weights8(ep, 4, 128, 128, 50)
    y, q, qs = torch.full((R, 128), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((R, 128), 5, dtype=torch.uint8, device="cuda"), torch.ones(R, 4, device="cuda")
    for _ in range(2):
        ep.ep_expert_gemm_f8(h, x, xs, w, ws, y)
        ep.ep_expert_dgrad_f8(h, x, xs, w, ws, y)
        ep.ep_expert_quantize(h, y, q.view(F8), qs)
        assert bool((y == 3.0).all()) and bool((q == 5).all()) and bool((qs == 1).all())
        ep.ep_prepare(h, torch.full((8, 2), -1, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda"), 1)  # every route masked


def test_offsets_past_2_to_the_31(ep):  # noqa: F811
    """The last expert's rows lie past element 2^31 of the rows, then of the gradients."""
    T, n, k = (1 << 18) + 96, 16, 8192
    lid, size = ep.ep_register_layer(2, 1, k, T, 1)
    R, h = ep.ep_recv_capacity(lid), ep.alloc_handle(lid, size)
    last = 90
    idx = torch.zeros(T, 1, dtype=torch.int64, device="cuda")
    idx[-last:] = 1
    ep.ep_prepare(h, idx, torch.empty(2, dtype=torch.int32, device="cuda"), 1)
    own = slice(T - last, T)
    x = torch.zeros(R, k, dtype=F8, device="cuda")
    xs = torch.zeros(R, columns(k), device="cuda")
    q, sc = torch.empty(last, k, dtype=F8, device="cuda"), torch.empty(last, columns(k), device="cuda")
    ep.ep_quantize_rows(wl.payload_normal(last, k, 51, "fp32").cuda(), q, sc)
    x.view(torch.uint8)[own], xs[own] = q.view(torch.uint8), sc
    w, ws, wv = weights8(ep, 2, n, k, 52)
    y = torch.empty(R, n, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_gemm_f8(h, x, xs, w, ws, y)
    v = q.double() * sc.double().repeat_interleave(128, 1)[:, :k]
    want, mag = v @ wv[1].t(), sum_bound(k) * (v.abs() @ wv[1].abs().t())
    assert bool(((y[own].double() - want).abs() <= mag + UNIT["bf16"] * (want.abs() + mag)).all())
    del x, xs
    dy, ds = torch.zeros(R, n, dtype=F8, device="cuda"), torch.zeros(R, columns(n), device="cuda")
    q, sc = torch.empty(last, n, dtype=F8, device="cuda"), torch.empty(last, columns(n), device="cuda")
    ep.ep_quantize_rows(wl.payload_normal(last, n, 53, "fp32").cuda(), q, sc)
    dy.view(torch.uint8)[own], ds[own] = q.view(torch.uint8), sc
    dx = torch.empty(R, k, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_dgrad_f8(h, dy, ds, w, ws, dx)
    v = q.double() * sc.double()[:, :1]
    want, mag = v @ wv[1], sum_bound(n) * (v.abs() @ wv[1].abs())
    assert bool(((dx[own].double() - want).abs() <= mag + UNIT["bf16"] * (want.abs() + mag)).all())
    assert bool((dx[: T - last: 4096] == 0).all())
