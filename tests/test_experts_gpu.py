"""Expert products against the same sums in 64 bits.

Tolerances.  A float32 sum of n products in any order, each operation rounded
by at most 2^-23 (the tensor core may truncate), is off by at most
n * 2^-23 * sum |a||b|; the result is then rounded once to the output type
(unit roundoff 2^-8 bf16, 2^-11 fp16, 2^-24 fp32; fp16 results below 2^-14
are rounded to multiples of 2^-24, half of that off).  The activation passes an
error on through its derivative (|silu'| <= 1.1) and adds its own, bounded by
2^-18 (1 + |gate|) of the terms it forms.
Rows that no expert owns (padding, and rows past the used ones) hold NaN in
every input, so anything read from them shows.
"""
import numpy as np
import pytest
import torch

from combine_ep_prepare_gb300 import workloads as wl
from tests.ep_harness import SENTINEL, SENTINEL32

pytestmark = pytest.mark.gpu

UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -120, "fp16": 2.0 ** -25, "fp32": 2.0 ** -120}
STEP = 2.0 ** -23
ACT = 2.0 ** -18


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import combine_ep_prepare_gb300 as ep
    return ep


def sentinel(rows, width, dtype):
    if dtype == "fp32":
        return torch.full((rows, width), SENTINEL32, dtype=torch.int32, device="cuda").view(torch.float32)
    return torch.full((rows, width), SENTINEL, dtype=torch.int16, device="cuda").view(wl.TORCH_PAYLOAD[dtype])


def is_sentinel(t):
    if t.dtype == torch.float32:
        return bool((t.view(torch.int32) == SENTINEL32).all())
    return bool((t.view(torch.int16) == SENTINEL).all())


class Step:
    """A prepared handle and where its rows are."""

    def __init__(self, ep, E, K, T, A, dtype, seed, p_mask=0.1, idx=None):
        self.E, self.dtype, self.tt = E, dtype, wl.TORCH_PAYLOAD[dtype]
        lid, size = ep.ep_register_layer(E, K, 64, T, A, dtype=dtype)
        self.R = ep.ep_recv_capacity(lid)
        self.h = ep.alloc_handle(lid, size)
        idx = wl.random_routing(T, K, E, seed, p_mask=p_mask)[0] if idx is None else idx
        counts = torch.empty(E, dtype=torch.int32, device="cuda")
        ep.ep_prepare(self.h, idx.cuda(), counts, A)
        off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        ep.ep_expert_offsets(self.h, off)
        self.counts, self.off = counts.tolist(), off.tolist()
        self.P = self.off[-1]
        self.spans = [(e, slice(self.off[e], self.off[e] + self.counts[e])) for e in range(E) if self.counts[e]]
        self.live = torch.zeros(self.R, dtype=torch.bool)
        for _, r in self.spans:
            self.live[r] = True
        self.pad = ~self.live
        self.pad[self.P:] = False

    def rows(self, width, seed, scale=1.0):
        x = (wl.payload_normal(self.R, width, seed, "fp32") * scale).to(self.tt)
        x[~self.live] = float("nan")
        return x.cuda()

    def weights(self, n, k, seed):
        return (wl.payload_normal(self.E * n, k, seed, "fp32") * k ** -0.5).to(self.tt).view(self.E, n, k).cuda()

    def out(self, width):
        return sentinel(self.R, width, self.dtype)

    def check_rows(self, got, want, bound):
        """want and bound: float64 [R, width] on the GPU, read in live rows."""
        got_cpu = got.cpu()
        assert is_sentinel(got[self.P:]), "rows past the used ones were written"
        assert bool((got_cpu[self.pad] == 0).all()), "padding rows are not zero"
        live = self.live.cuda()
        d = (got[live].double() - want[live]).abs()
        assert bool(torch.isfinite(got[live]).all())
        worst = (d / (bound[live] + TINY[self.dtype])).max().item() if d.numel() else 0.0
        assert worst <= 1.0, "error %.3g of its bound" % worst

    def per_row(self, fn, width):
        """Two float64 [R, width]: fn(e, rows) -> (value, magnitude of the sum's terms)."""
        v = torch.zeros(self.R, width, dtype=torch.float64, device="cuda")
        m = torch.zeros_like(v)
        for e, r in self.spans:
            v[r], m[r] = fn(e, r)
        return v, m


def product(x, w):
    x, w = x.double(), w.double()
    return x @ w, x.abs() @ w.abs()


# E, K, T, A, in, out: one token, one expert, empty experts, ragged ends in every dimension, alignments
# that are no tile's, an expert with several row tiles, batches with a row block of padding alone.
SHAPES = [(1, 1, 1, 1, 8, 8), (8, 2, 1, 128, 64, 72), (4, 1, 3, 1, 200, 136), (64, 2, 40, 1, 72, 264),
          (8, 2, 700, 128, 256, 264), (3, 2, 500, 300, 136, 520), (16, 4, 333, 7, 520, 128),
          (2, 1, 1030, 16, 1032, 776), (300, 3, 200, 4, 64, 48), (5, 2, 64, 1, 1024, 2048)]
TYPES = ["bf16", "fp16", "fp32"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gemm(ep, shape, dtype):
    E, K, T, A, n_in, n_out = shape
    s = Step(ep, E, K, T, A, dtype, 1)
    x, w, y = s.rows(n_in, 11), s.weights(n_out, n_in, 12), s.out(n_out)
    ep.ep_expert_gemm(s.h, x, w, y)
    want, mag = s.per_row(lambda e, r: product(x[r], w[e].t()), n_out)
    s.check_rows(y, want, n_in * STEP * mag + UNIT[dtype] * want.abs())


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gemm_swiglu(ep, shape, dtype, keep):
    E, K, T, A, n_in, f = shape
    s = Step(ep, E, K, T, A, dtype, 2)
    x, w, act = s.rows(n_in, 21), s.weights(2 * f, n_in, 22), s.out(f)
    pre = s.out(2 * f) if keep else None
    ep.ep_expert_gemm_swiglu(s.h, x, w, act, pre=pre)
    want, mag = s.per_row(lambda e, r: product(x[r], w[e].t()), 2 * f)
    err = n_in * STEP * mag
    if keep:
        s.check_rows(pre, want, err + UNIT[dtype] * want.abs())
    g, u = want[:, :f], want[:, f:]
    silu = torch.nn.functional.silu(g)
    bound = 1.1 * err[:, :f] * (u.abs() + err[:, f:]) + silu.abs() * err[:, f:]
    bound = bound + (ACT * (1 + g.abs()) + UNIT[dtype]) * (silu * u).abs()
    s.check_rows(act, silu * u, bound)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dgrad(ep, shape, dtype):
    E, K, T, A, n_in, n_out = shape
    s = Step(ep, E, K, T, A, dtype, 3)
    dy, w, dx = s.rows(n_out, 31), s.weights(n_out, n_in, 32), s.out(n_in)
    ep.ep_expert_dgrad(s.h, dy, w, dx)
    want, mag = s.per_row(lambda e, r: product(dy[r], w[e]), n_in)
    s.check_rows(dx, want, n_out * STEP * mag + UNIT[dtype] * want.abs())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dgrad_swiglu(ep, shape, dtype):
    E, K, T, A, f, n_out = shape
    s = Step(ep, E, K, T, A, dtype, 4)
    dy, w, pre, dpre = s.rows(n_out, 41), s.weights(n_out, f, 42), s.rows(2 * f, 43, 3.0), s.out(2 * f)
    ep.ep_expert_dgrad_swiglu(s.h, dy, w, pre, dpre)
    da, mag = s.per_row(lambda e, r: product(dy[r], w[e]), f)
    p = torch.nan_to_num(pre.double()).requires_grad_()
    act = torch.nn.functional.silu(p[:, :f]) * p[:, f:]
    want = torch.autograd.grad(act, p, da)[0]
    g, u = p.detach()[:, :f], p.detach()[:, f:]
    sg = torch.sigmoid(g)
    slope = torch.cat([u * sg * (1 + g * (1 - sg)), g * sg], 1).abs()
    terms = torch.cat([u.abs() * sg * (1 + g.abs()), g.abs() * sg], 1)
    err, da2, g2 = (torch.cat([t, t], 1) for t in (n_out * STEP * mag, da.abs(), g.abs()))
    s.check_rows(dpre, want, slope * err + ACT * (1 + g2) * terms * (da2 + err) + UNIT[dtype] * want.abs())


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype,wtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                         ("fp32", "fp32")])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_wgrad(ep, shape, dtype, wtype, accumulate):
    E, K, T, A, n_in, n_out = shape
    s = Step(ep, E, K, T, A, dtype, 5)
    dy, x = s.rows(n_out, 51), s.rows(n_in, 52)
    if accumulate:
        dw = wl.payload_normal(E * n_out, n_in, 53, wtype).view(E, n_out, n_in).cuda()
        want = dw.double()
    else:
        dw = sentinel(E * n_out, n_in, wtype).view(E, n_out, n_in)
        want = torch.zeros(E, n_out, n_in, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    before = dw.clone()
    for e, r in s.spans:
        v, m = product(dy[r].t(), x[r])
        want[e] += v
        bound[e] = s.counts[e] * STEP * m
    bound += (UNIT[wtype] + (2.0 ** -24 if accumulate else 0.0)) * (want.abs() + bound) + TINY[wtype]
    ep.ep_expert_wgrad(s.h, dy, x, dw, accumulate=accumulate)
    empty = [e for e in range(E) if not s.counts[e]]
    assert torch.equal(dw[empty], before[empty] if accumulate else torch.zeros_like(dw[empty]))
    d = (dw.double() - want).abs()
    assert bool((d <= bound).all()), (d / bound).max().item()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_long_float32_gradients_keep_their_precision(ep, dtype, accumulate):
    """Weight gradients over thousands of rows in float32, against the norm of
    the result.  The tensor core truncates: 20,000 rows in one sum would be
    off by 2e-5.  The tolerance is that of sums of 512 rows (32 accumulations,
    at most 2^-23 each), the 40 of them added in float32 with rounding to
    nearest (at most 2^-24 each): 6.2e-6."""
    s = Step(ep, 3, 1, 24000, 1, dtype, 13, p_mask=0.0, idx=(torch.arange(24000) % 12).clamp(max=2).view(-1, 1))
    assert s.counts == [2000, 2000, 20000]
    dy, x = s.rows(72, 71), s.rows(136, 72)
    dw = torch.zeros(3, 72, 136, device="cuda")
    if accumulate:
        dw = wl.payload_normal(3 * 72, 136, 73, "fp32").view(3, 72, 136).cuda()
    before = dw.double()
    ep.ep_expert_wgrad(s.h, dy, x, dw, accumulate=accumulate)
    for e, r in s.spans:
        want = dy[r].double().t() @ x[r].double() + (before[e] if accumulate else 0)
        assert ((dw[e].double() - want).norm() / want.norm()).item() <= 32 * 2.0 ** -23 + 40 * 2.0 ** -24


@pytest.mark.parametrize("dtype", TYPES)
def test_no_tokens(ep, dtype):
    s = Step(ep, 4, 2, 0, 16, dtype, 6)
    assert s.P == 0
    x, w, y = s.rows(64, 1), s.weights(72, 64, 2), s.out(72)
    dw = sentinel(4 * 72, 64, dtype).view(4, 72, 64)
    # a capacity of no rows at all leaves nothing to address: no row buffer of the wrong size is read
    ep.ep_expert_gemm(s.h, torch.empty(1, 64, dtype=s.tt, device="cuda"), w, torch.empty(1, 72, dtype=s.tt, device="cuda"))
    ep.ep_expert_wgrad(s.h, torch.empty(1, 72, dtype=s.tt, device="cuda"), torch.empty(1, 64, dtype=s.tt, device="cuda"), dw)
    torch.cuda.synchronize()
    assert bool((dw == 0).all())
    assert x.numel() == 0 and y.numel() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_all_routes_masked(ep, dtype):
    s = Step(ep, 4, 2, 20, 16, dtype, 7, idx=torch.full((20, 2), -1, dtype=torch.int64))
    x, w, y = s.rows(64, 1), s.weights(72, 64, 2), s.out(72)
    ep.ep_expert_gemm(s.h, x, w, y)
    dw = sentinel(4 * 72, 64, dtype).view(4, 72, 64)
    ep.ep_expert_wgrad(s.h, s.rows(72, 3), x, dw)
    assert is_sentinel(y) and bool((dw == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_unprepared_and_overflowed_handles_write_nothing(ep, dtype):
    lid, size = ep.ep_register_layer(4, 2, 64, 32, 16, recv_capacity=40, dtype=dtype)
    tt = wl.TORCH_PAYLOAD[dtype]
    x, w = torch.ones(40, 64, dtype=tt, device="cuda"), torch.ones(4, 64, 64, dtype=tt, device="cuda")
    dw = sentinel(4 * 64, 64, dtype).view(4, 64, 64)
    h = ep.alloc_handle(lid, size)
    for prepare in (False, True):
        if prepare:
            counts = torch.empty(4, dtype=torch.int32, device="cuda")
            ep.ep_prepare(h, wl.random_routing(32, 2, 4, 3)[0].cuda(), counts, 16)
            assert ep.ep_read_info(h)["status"] & ep.EP_ST_OVERFLOW
        y = sentinel(40, 64, dtype)
        ep.ep_expert_gemm(h, x, w, y)
        ep.ep_expert_dgrad(h, x, w, y)
        ep.ep_expert_wgrad(h, x, x, dw)
        if dtype != "fp32":
            wq, sc = torch.zeros(4, 64, 32, dtype=torch.uint8, device="cuda"), torch.ones(4, 64, 2, dtype=tt, device="cuda")
            ep.ep_expert_gemv_w4(h, x, wq, sc, y)
        assert is_sentinel(y) and is_sentinel(dw)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nan_and_infinity_stay_with_their_expert(ep, dtype):
    """A non-finite weight or row of one expert shows in that expert alone."""
    s = Step(ep, 6, 2, 150, 1, dtype, 8, p_mask=0.0)
    x, w = s.rows(136, 1), s.weights(200, 136, 2)
    w[2] = float("inf")
    x[s.spans[4][1]] = float("nan")
    y, dx = s.out(200), s.out(136)
    ep.ep_expert_gemm(s.h, x, w, y)
    ep.ep_expert_dgrad(s.h, y, w, dx)
    dw = sentinel(6 * 200, 136, dtype).view(6, 200, 136)
    ep.ep_expert_wgrad(s.h, y, x, dw)
    for e, r in s.spans:
        bad = e in (2, 4)
        assert bool(torch.isfinite(y[r]).all()) != bad
        assert bool(torch.isfinite(dx[r]).all()) != bad
        assert bool(torch.isfinite(dw[e]).all()) != bad


@pytest.mark.parametrize("value", [float("inf"), float("nan")], ids=["inf", "nan"])
@pytest.mark.parametrize("dtype", TYPES)
def test_padding_rows_are_zero_whatever_the_weights_hold(ep, dtype, value):
    """0 * inf is NaN, so a padding row must not be what a product with its zeros gives."""
    s = Step(ep, 5, 2, 70, 100, dtype, 81)
    x, dy = s.rows(96, 82), s.rows(160, 83)
    w, w13 = s.weights(160, 96, 84), s.weights(144, 96, 85)
    w[:, 3, 5], w13[:, 7, 9], w13[:, 80, 11] = value, value, value
    y, act, dx, dpre = s.out(160), s.out(72), s.out(96), s.out(192)
    ep.ep_expert_gemm(s.h, x, w, y)
    ep.ep_expert_gemm_swiglu(s.h, x, w13, act)
    ep.ep_expert_dgrad(s.h, dy, w, dx)
    ep.ep_expert_dgrad_swiglu(s.h, dy, w, s.rows(192, 86), dpre)
    outs = [y, act, dx, dpre]
    if dtype != "fp32":
        wq, scales, _ = w4_weights(s, 80, 96, 32, 87)
        scales[:, 2, 1] = value
        outs.append(s.out(80))
        ep.ep_expert_gemv_w4(s.h, x, wq, scales, outs[-1])
    assert bool(s.pad.any())
    for o in outs:
        assert bool((o.cpu()[s.pad] == 0).all())
        assert is_sentinel(o[s.P:])


@pytest.mark.parametrize("dtype", TYPES)
def test_same_inputs_same_bits_and_other_stream(ep, dtype):
    s = Step(ep, 8, 2, 300, 16, dtype, 9)
    x, w = s.rows(264, 1), s.weights(392, 264, 2)
    side = torch.cuda.Stream()
    outs = []
    for stream in (None, side, side):
        y, dw = s.out(392), torch.zeros(8, 392, 264, dtype=torch.float32, device="cuda")
        torch.cuda.synchronize()
        ep.ep_expert_gemm(s.h, x, w, y, stream=stream)
        ep.ep_expert_wgrad(s.h, y, x, dw, accumulate=True, stream=stream)
        torch.cuda.synchronize()
        outs.append((y, dw))
    for y, dw in outs[1:]:
        assert torch.equal(y[s.live.cuda()], outs[0][0][s.live.cuda()]) and torch.equal(dw, outs[0][1])


@pytest.mark.parametrize("dtype", TYPES)
def test_captured_products_follow_a_new_routing(ep, dtype):
    """One graph of prepare, dispatch and the products, replayed on another routing in the same buffers."""
    E, K, T, A, H, F = 8, 2, 260, 16, 136, 72
    tt = wl.TORCH_PAYLOAD[dtype]
    lid, size = ep.ep_register_layer(E, K, H, T, A, dtype=dtype)
    R = ep.ep_recv_capacity(lid)
    h = ep.alloc_handle(lid, size)
    idx = wl.random_routing(T, K, E, 1)[0].cuda()
    wts = wl.random_routing(T, K, E, 1)[1].cuda()
    tok = wl.payload_normal(T, H, 5, dtype).cuda()
    w = (wl.payload_normal(E * 2 * F, H, 6, "fp32") * H ** -0.5).to(tt).view(E, 2 * F, H).cuda()
    recv, rw = torch.zeros(R, H, dtype=tt, device="cuda"), torch.zeros(R, device="cuda")
    act, counts = torch.zeros(R, F, dtype=tt, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda")

    def step():
        ep.ep_prepare(h, idx, counts, A)
        ep.ep_dispatch(h, idx, tok, wts, recv, rw)
        ep.ep_expert_gemm_swiglu(h, recv, w, act)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2, 3):
        idx.copy_(wl.random_routing(T, K, E, seed, p_mask=0.2)[0])
        g.replay()
        torch.cuda.synchronize()
        replayed = act.clone()
        used = ep.ep_read_info(h)["used_rows"]
        step()
        torch.cuda.synchronize()
        assert torch.equal(replayed[:used], act[:used])
        slots = torch.empty(T, K, dtype=torch.int32, device="cuda")
        ep.ep_token_slots(h, slots)
        t, k = 17, int((idx[17] >= 0).nonzero()[0])
        pre = w[idx[t, k]].double() @ tok[t].double()
        want = torch.nn.functional.silu(pre[:F]) * pre[F:]
        assert (replayed[slots[t, k]].double() - want).abs().max() <= 4 * UNIT[dtype] * want.abs().max() + H * STEP * 40


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sharded_owner(ep, dtype):
    """A sharded layer's products run on its own experts."""
    E, K, T, N, A, n_in, n_out = 8, 2, 100, 2, 8, 72, 136
    tt = wl.TORCH_PAYLOAD[dtype]
    idx = [wl.random_routing(T, K, E, 70 + r, p_mask=0.1)[0].cuda() for r in range(N)]
    hs, local = [], []
    for r in range(N):
        lid, size = ep.ep_register_layer_sharded(E, K, 64, T, N, r, A, dtype=dtype)
        R = ep.ep_recv_capacity(lid)
        hs.append(ep.alloc_handle(lid, size))
        local.append(torch.empty(E, dtype=torch.int32, device="cuda"))
        ep.ep_shard_count(hs[r], idx[r], local[r])
    table = torch.stack(local)
    for r in range(N):
        counts = torch.empty(E // N, dtype=torch.int32, device="cuda")
        ep.ep_shard_prepare(hs[r], idx[r], table, counts, A)
        off = torch.empty(E // N + 1, dtype=torch.int32, device="cuda")
        ep.ep_expert_offsets(hs[r], off)
        x = wl.payload_normal(R, n_in, 5, dtype).cuda()
        w = wl.payload_normal(E // N * n_out, n_in, 6, dtype).view(E // N, n_out, n_in).cuda()
        y = sentinel(R, n_out, dtype)
        ep.ep_expert_gemm(hs[r], x, w, y)
        dw = torch.empty_like(w)
        ep.ep_expert_wgrad(hs[r], torch.nan_to_num(y), x, dw)
        off, counts = off.tolist(), counts.tolist()
        assert is_sentinel(y[off[-1]:])
        for e in range(E // N):
            rows = slice(off[e], off[e] + counts[e])
            want, mag = product(x[rows], w[e].t())
            assert bool(((y[rows].double() - want).abs() <= n_in * STEP * mag + UNIT[dtype] * want.abs()).all())
            assert bool((y[off[e] + counts[e]:off[e + 1]] == 0).all())
            want, mag = product(y[rows].t(), x[rows])
            assert bool(((dw[e].double() - want).abs() <= (counts[e] * STEP + UNIT[dtype]) * mag).all())


def test_gradients_against_differences(ep):
    """The gradients of a loss over gate/up, activation and down products, in
    fp32, along random directions.  A central difference with step h of a
    smooth loss is off by O(h^2) of its third derivative; with h = 2^-6 and
    inputs of size 1 that and the float32 noise (2^-24 * loss / h) stay under
    2% of the size of a directional derivative."""
    E, K, T, A, H, F = 4, 2, 60, 4, 40, 24
    s = Step(ep, E, K, T, A, "fp32", 10)
    x, w13, w2, gy = s.rows(H, 1), s.weights(2 * F, H, 2), s.weights(H, F, 3), s.rows(H, 4)
    live = s.live.cuda()

    def loss(x, w13, w2):
        pre, act, y = s.out(2 * F), s.out(F), s.out(H)
        ep.ep_expert_gemm_swiglu(s.h, x, w13, act, pre=pre)
        ep.ep_expert_gemm(s.h, act, w2, y)
        return (y[live].double() * gy[live].double()).sum().item(), pre, act

    _, pre, act = loss(x, w13, w2)
    dpre, dx, dw13, dw2 = s.out(2 * F), s.out(H), torch.empty_like(w13), torch.empty_like(w2)
    ep.ep_expert_dgrad_swiglu(s.h, gy, w2, pre, dpre)
    ep.ep_expert_wgrad(s.h, gy, act, dw2)
    ep.ep_expert_dgrad(s.h, dpre, w13, dx)
    ep.ep_expert_wgrad(s.h, dpre, x, dw13)
    step = 2.0 ** -6
    for name, i, grad in (("x", 0, dx), ("w13", 1, dw13), ("w2", 2, dw2)):
        args = [x, w13, w2]
        g = torch.Generator().manual_seed(90 + i)
        d = torch.randn(args[i].shape, generator=g).cuda() * args[i].isfinite()
        d = d / d.norm() * (2 * d.shape[-1]) ** 0.5
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * d, args[i] - step * d
        diff = (loss(*up)[0] - loss(*down)[0]) / (2 * step)
        G = torch.where(args[i].isfinite(), grad, torch.zeros_like(grad)).double()
        want = (G * d.double()).sum().item()
        size = (G.norm() * d.double().norm()).item() / np.sqrt(d.numel())
        assert abs(diff - want) <= 0.02 * max(abs(want), size), (name, diff, want)


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------

# E, K, T, A, in, out, group
W4_SHAPES = [(1, 1, 1, 1, 32, 8, 32), (8, 2, 1, 1, 128, 72, 64), (8, 4, 5, 8, 256, 264, 128), (16, 2, 60, 1, 384, 40, 32),
             (2, 2, 77, 16, 1152, 136, 128), (40, 8, 33, 1, 2048, 24, 64), (4, 1, 300, 5, 640, 56, 128),
             (3, 1, 9, 1, 7168, 520, 128), (64, 8, 1, 1, 1024, 1024, 32)]


def w4_weights(s, n, k, group, seed):
    g = torch.Generator().manual_seed(seed)
    wq = torch.randint(0, 256, (s.E, n, k // 2), generator=g, dtype=torch.uint8)
    sc = ((0.5 + torch.rand(s.E, n, k // group, generator=g)) * k ** -0.5).to(s.tt)
    q = torch.stack([wq & 15, wq >> 4], dim=3).flatten(2).double() - 8
    return wq.cuda(), sc.cuda(), (q * sc.double().repeat_interleave(group, dim=2)).cuda()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", W4_SHAPES, ids=str)
def test_gemv_w4(ep, shape, dtype, gated):
    E, K, T, A, n_in, n_out, group = shape
    s = Step(ep, E, K, T, A, dtype, 11)
    x = s.rows(n_in, 61)
    wq, sc, w = w4_weights(s, 2 * n_out if gated else n_out, n_in, group, 62)
    y = s.out(n_out)
    (ep.ep_expert_gemv_w4_swiglu if gated else ep.ep_expert_gemv_w4)(s.h, x, wq, sc, y)
    want, mag = s.per_row(lambda e, r: product(x[r], w[e].t()), w.shape[1])
    err = (n_in + 2) * STEP * mag
    if gated:
        g, u = want[:, :n_out], want[:, n_out:]
        silu = torch.nn.functional.silu(g)
        err = 1.1 * err[:, :n_out] * (u.abs() + err[:, n_out:]) + silu.abs() * err[:, n_out:]
        want = silu * u
        err = err + ACT * (1 + g.abs()) * want.abs()
    s.check_rows(y, want, err + UNIT[dtype] * want.abs())


def test_gemv_w4_nonfinite_rows_and_scales_stay_put(ep):
    s = Step(ep, 4, 2, 30, 1, "bf16", 12, p_mask=0.0)
    wq, sc, _ = w4_weights(s, 72, 256, 64, 5)
    x = s.rows(256, 1)
    sc[1] = float("nan")
    first = s.spans[3][1].start
    x[first] = float("inf")
    y = s.out(72)
    ep.ep_expert_gemv_w4(s.h, x, wq, sc, y)
    for e, r in s.spans:
        rows = torch.isfinite(y[r]).all(dim=1)
        if e == 1:
            assert not bool(rows.any())
        elif e == 3:
            assert not bool(rows[0]) and bool(rows[1:].all())
        else:
            assert bool(rows.all())


def test_pack_w4_round_trip(ep):
    w = (wl.payload_normal(3 * 40, 256, 8, "fp32") * 0.1).to(torch.bfloat16).view(3, 40, 256)
    w[1, 5, 64:128] = 0
    wq, sc = ep.pack_w4(w, 64)
    q = torch.stack([wq & 15, wq >> 4], dim=3).flatten(2).float() - 8
    back = q * sc.float().repeat_interleave(64, dim=2)
    # half a step, and what the rounded scale leaves beyond the largest code
    assert bool(((back - w.float()).abs() <= sc.float().repeat_interleave(64, dim=2) * 0.54).all())
    assert bool((back[1, 5, 64:128] == 0).all())
