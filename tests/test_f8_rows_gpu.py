"""The norm, its gradient, the quantisation of rows and their dispatch.

Tolerances.  The norm's sum of H squares and the two means of its gradient are
float32 sums of positive or of signed terms in some tree: at most (H / threads
+ 16) <= 64 additions deep, each off by 2^-24 of the sum of magnitudes; a
quotient, a square root and four products add 8 * 2^-24.  So r is off by at
most (64 / 2 + 8) 2^-24 < 2.4e-6 of itself, y by 3e-6, and a result is then
rounded once to its type (2^-8, 2^-11, 2^-24 of the value).  Quantised values
of given rows are compared bit for bit with the float32 formula.
"""
import pytest
import torch

from combine_ep_prepare_gb300 import workloads as wl
from tests.test_experts_gpu import TINY, UNIT, Step, ep  # noqa: F401

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
Y = 3e-6


def columns(n):
    return ((n + 127) // 128 + 3) // 4 * 4


def quantize(x):
    """The float32 formula, on the CPU: (q, scales padded to a multiple of four)."""
    T, n = x.shape
    b = torch.nn.functional.pad(x.float().cpu(), (0, (n + 127) // 128 * 128 - n)).view(T, -1, 128)
    m = b.abs().amax(2).clamp_min(2.0 ** -100)
    q = (b * (torch.full_like(m, 448.0) / m)[:, :, None]).clamp(-448, 448).to(F8).view(T, -1)[:, :n]
    return q.contiguous(), torch.nn.functional.pad(m / torch.full_like(m, 448.0), (0, columns(n) - m.shape[1]))


def same(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


def rows(T, n, seed, dtype, spread=True):
    x = wl.payload_normal(T, n, seed, "fp32")
    if spread:  # blocks of very different magnitude
        x = x * torch.logspace(-3, 2, (n + 127) // 128).repeat_interleave(128)[:n]
    return x.to(wl.TORCH_PAYLOAD[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,n", [(1, 16), (3, 128), (7, 144), (33, 2064), (129, 1024), (1, 32768)])
def test_quantize_rows_bit_for_bit(ep, T, n, dtype):  # noqa: F811
    x = rows(T, n, 5, dtype)
    if T > 2:
        x[1] = 0                                       # a row of zeros
        x[2, : min(n, 100)] = torch.finfo(x.dtype).tiny  # the type's smallest
        x[0, n // 2] = torch.finfo(x.dtype).max / 4
    q, s = torch.empty(T, n, dtype=F8, device="cuda"), torch.full((T, columns(n)), float("nan"), device="cuda")
    ep.ep_quantize_rows(x, q, s)
    wq, ws = quantize(x)
    assert same(q, wq) and torch.equal(s.cpu(), ws)


def test_quantize_marks_blocks_without_finite_values(ep):  # noqa: F811
    x = rows(4, 384, 6, "bf16")
    x[0, 5], x[1, 200], x[2, 383] = float("nan"), float("inf"), -float("inf")
    q, s = torch.empty(4, 384, dtype=F8, device="cuda"), torch.empty(4, 4, device="cuda")
    ep.ep_quantize_rows(x, q, s)
    value = (q.float() * s.repeat_interleave(128, 1)[:, :384]).view(4, 3, 128)
    bad = torch.zeros(4, 3, dtype=torch.bool)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert torch.equal(torch.isnan(value).all(2).cpu(), bad) and torch.equal(torch.isnan(value).any(2).cpu(), bad)


def norm_reference(x, res, w, eps):
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    r = torch.rsqrt(h.double().square().mean(1, keepdim=True) + eps)
    return h, h.double() * r * w.double(), r


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", [(1, 16), (2, 80), (5, 128), (33, 1040), (130, 2048), (64, 7168), (3, 8208), (2, 32768)])
def test_norm(ep, T, H, residual, dtype):  # noqa: F811
    x, res = rows(T, H, 7, dtype, spread=False), rows(T, H, 8, dtype, spread=False) if residual else None
    w = (1 + 0.3 * wl.payload_normal(1, H, 9, "fp32")[0]).to(x.dtype).cuda()
    y, total = torch.empty_like(x), torch.empty_like(x) if residual else None
    q, s = torch.empty(T, H, dtype=F8, device="cuda"), torch.full((T, columns(H)), float("nan"), device="cuda")
    ep.ep_rmsnorm(x, w, y=y, residual=res, sum=total, q=q, scales=s, eps=1e-5)
    h, want, _ = norm_reference(x, res, w, 1e-5)
    if residual:
        assert torch.equal(total, h)
    assert bool(((y.double() - want).abs() <= (UNIT[dtype] + Y) * want.abs() + TINY[dtype]).all())
    blocks = torch.nn.functional.pad(want, (0, -H % 128)).view(T, -1, 128)
    m = blocks.abs().amax(2) / 448
    assert bool(((s[:, :m.shape[1]].double() - m).abs() <= 2 * Y * m).all()) and bool((s[:, m.shape[1]:] == 0).all())
    v = (blocks / m[:, :, None]).view(T, -1)[:, :H]
    assert bool(((q.double() - v).abs() <= v.abs() * (2.0 ** -4 + 4 * Y) + 2.0 ** -10).all())
    # each result alone, and in place
    y2, total2 = x.clone(), None
    ep.ep_rmsnorm(y2, w, y=y2, residual=res, eps=1e-5)
    assert torch.equal(y2, y)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    ep.ep_rmsnorm(x, w, residual=res, q=q2, scales=s2, eps=1e-5)
    assert same(q2, q) and torch.equal(s2, s)
    if residual:
        total2 = res.clone()
        ep.ep_rmsnorm(x, w, residual=total2, sum=total2, eps=1e-5)
        assert torch.equal(total2, total)


def test_norm_of_zero_rows_and_no_tokens(ep):  # noqa: F811
    x, w = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda"), torch.ones(256, dtype=torch.bfloat16, device="cuda")
    y, q, s = torch.empty_like(x), torch.empty(3, 256, dtype=F8, device="cuda"), torch.empty(3, 4, device="cuda")
    ep.ep_rmsnorm(x, w, y=y, q=q, scales=s)
    assert bool((y == 0).all()) and bool((q.float() == 0).all()) and bool(torch.isfinite(s).all())
    before = ep.ep_launch_count()
    ep.ep_rmsnorm(x[:0], w, y=y[:0])
    assert ep.ep_launch_count() == before


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("through", [False, True])
@pytest.mark.parametrize("T,H", [(1, 8), (2, 80), (5, 1024), (700, 200), (1001, 2176), (40, 7168), (5, 8208), (310, 16384), (3, 32768)])
def test_norm_gradient(ep, T, H, through, dtype):  # noqa: F811
    eps = 1e-5
    h, dy = rows(T, H, 10, dtype, spread=False), rows(T, H, 11, dtype, spread=False)
    ds = rows(T, H, 12, dtype, spread=False) if through else None
    w = (1 + 0.3 * wl.payload_normal(1, H, 13, "fp32")[0]).to(h.dtype).cuda()
    dh, dw, work = torch.empty_like(h), torch.empty(H, device="cuda"), ep.rmsnorm_bwd_workspace(T, H)
    work.fill_(0xff)  # NaN: nothing is expected there
    ep.ep_rmsnorm_bwd(dy, h, w, dh, dw, work, grad_sum=ds, eps=eps)
    hh, ww = h.double().requires_grad_(), w.double().requires_grad_()
    y = hh * torch.rsqrt(hh.square().mean(1, keepdim=True) + eps) * ww
    gh, gw = torch.autograd.grad(y, (hh, ww), dy.double())
    with torch.no_grad():
        r = torch.rsqrt(hh.square().mean(1, keepdim=True) + eps)
        terms = r * ((ww * dy.double()).abs() + hh.abs() * r * r * (ww * dy.double() * hh).abs().mean(1, keepdim=True))
        want = gh + (ds.double() if through else 0)
        bound = UNIT[dtype] * want.abs() + 8e-6 * terms + 2.0 ** -23 * want.abs() + TINY[dtype]
        assert bool(((dh.double() - want).abs() <= bound).all())
        # T terms, each off by 3e-6 and added in at most T / parts + parts / 16 + 16 <= 64 steps of 2^-24 (152 to 608 parts)
        mag = (dy.double() * hh * r).abs().sum(0)
        assert bool(((dw.double() - gw).abs() <= 8e-6 * mag + 1e-37).all())
    again, dw2 = dy.clone(), dw.clone()
    ep.ep_rmsnorm_bwd(again, h, w, again, dw2, work, grad_sum=ds, eps=eps, accumulate=True)  # in place, added to
    assert torch.equal(again, dh) and torch.equal(dw2, dw + dw)


def test_norm_gradient_of_no_tokens(ep):  # noqa: F811
    h, w, dw = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda"), torch.full((64,), 3.0, device="cuda")
    work = ep.rmsnorm_bwd_workspace(0, 64)
    ep.ep_rmsnorm_bwd(h, h, w, h.clone(), dw, work, accumulate=True)
    assert bool((dw == 3).all())
    ep.ep_rmsnorm_bwd(h, h, w, h.clone(), dw, work)
    assert bool((dw == 0).all())


def test_norm_gradient_against_differences(ep):  # noqa: F811
    """<dy, y(h + d) - y(h - d)> / 2 against <dh, d>, and the same for the
    weight.  With |d| about 2^-6 |h| the third-order term is 2^-12 of the first
    order's magnitude, float32's rounding of y, 2^-23 of it, over 2^-6 less."""
    T, H = 6, 256
    h, dy, d = rows(T, H, 14, "fp32", False), rows(T, H, 15, "fp32", False), rows(T, H, 16, "fp32", False) * 2.0 ** -6
    w, dwn = 1 + 0.3 * rows(1, H, 17, "fp32", False)[0], rows(1, H, 18, "fp32", False)[0] * 2.0 ** -6
    dh, dw, work = torch.empty_like(h), torch.empty(H, device="cuda"), ep.rmsnorm_bwd_workspace(T, H)
    ep.ep_rmsnorm_bwd(dy, h, w, dh, dw, work)

    def f(a, b):
        y = torch.empty_like(a)
        ep.ep_rmsnorm(a.contiguous(), b.contiguous(), y=y)
        return (y.double() * dy.double()).sum()

    size = (dy.double() * d.double()).abs().sum()
    assert abs((f(h + d, w) - f(h - d, w)) / 2 - (dh.double() * d.double()).sum()) <= 2.0 ** -11 * 4 * size
    assert abs((f(h, w + dwn) - f(h, w - dwn)) / 2 - (dw.double() * dwn.double()).sum()) <= 2.0 ** -11 * 4 * size


@pytest.mark.parametrize("A", [1, 16])
@pytest.mark.parametrize("E,K,T,n,p_mask", [(8, 2, 40, 256, 0.1), (300, 8, 64, 1040, 0.3), (3, 1, 5, 16, 0.0), (4, 2, 9, 128, 1.0)])
def test_expert_quantize_leaves_other_rows(ep, E, K, T, n, A, p_mask):  # noqa: F811
    s = Step(ep, E, K, T, A, "bf16", 20, p_mask=p_mask)
    x = s.rows(n, 21)
    q = torch.full((s.R, n), 0x35, dtype=torch.uint8, device="cuda").view(F8)
    sc = torch.full((s.R, columns(n)), 7.0, device="cuda")
    ep.ep_expert_quantize(s.h, x, q, sc)
    wq, ws = quantize(x)
    q, sc = q.view(torch.uint8).cpu(), sc.cpu()
    assert torch.equal(q[s.live], wq.view(torch.uint8)[s.live]) and torch.equal(sc[s.live], ws[s.live])
    assert bool((q[s.pad] == 0).all()) and bool((sc[s.pad] == 0).all())
    assert bool((q[s.P:] == 0x35).all()) and bool((sc[s.P:] == 7.0).all())


@pytest.mark.parametrize("A", [1, 16])
@pytest.mark.parametrize("E,K,T,H,p_mask", [(8, 2, 40, 256, 0.1), (64, 8, 128, 7168, 0.5), (300, 8, 64, 1040, 0.3), (3, 1, 5, 16, 0.0),
                                            (4, 2, 9, 528, 1.0), (2, 2, 2000, 2048, 0.0), (4, 2, 3001, 2080, 0.2), (4, 2, 1500, 2064, 0.2),
                                            (2, 1, 2500, 16, 0.0)])
def test_dispatch_f8(ep, E, K, T, H, A, p_mask):  # noqa: F811
    idx, wts = wl.random_routing(T, K, E, 22, p_mask=p_mask)
    lid, size = ep.ep_register_layer(E, K, H, T, A)
    R, h = ep.ep_recv_capacity(lid), ep.alloc_handle(lid, size)
    counts, off = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    idx, wts = idx.cuda(), wts.cuda()
    ep.ep_prepare(h, idx, counts, A)
    slots = torch.empty(T, K, dtype=torch.int32, device="cuda")
    ep.ep_token_slots(h, slots)
    ep.ep_expert_offsets(h, off)
    P = int(off[-1])
    x = rows(T, H, 23, "bf16")
    q, s = torch.empty(T, H, dtype=F8, device="cuda"), torch.empty(T, columns(H), device="cuda")
    ep.ep_quantize_rows(x, q, s)
    rq = torch.full((R, H), 0x35, dtype=torch.uint8, device="cuda")
    rs, rw = torch.full((R, columns(H)), 7.0, device="cuda"), torch.full((R,), 7.0, device="cuda")
    ep.ep_dispatch_f8(h, idx, q, s, wts, rq.view(F8), rs, rw)
    wq, wsc, ww = torch.zeros(P, H, dtype=torch.uint8, device="cuda"), torch.zeros(P, columns(H), device="cuda"), torch.zeros(P, device="cuda")
    t, k = (slots >= 0).nonzero(as_tuple=True)
    at = slots[t, k].long()
    wq[at], wsc[at], ww[at] = q.view(torch.uint8)[t], s[t], wts[t, k]
    assert torch.equal(rq[:P], wq) and torch.equal(rs[:P], wsc) and torch.equal(rw[:P], ww)
    assert bool((rq[P:] == 0x35).all()) and bool((rs[P:] == 7.0).all()) and bool((rw[P:] == 7.0).all())


def test_offsets_past_2_to_the_31(ep):  # noqa: F811
    """The last rows of tensors with more than 2^31 elements are those of a call on them alone."""
    T, H, n = (1 << 18) + 40, 8192, 4
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(24))
    w = (1 + 0.3 * rows(1, H, 25, "bf16", False)[0]).to(x.dtype)
    q, s = torch.empty(T, H, dtype=F8, device="cuda"), torch.empty(T, columns(H), device="cuda")
    q2, s2 = torch.empty(n, H, dtype=F8, device="cuda"), torch.empty(n, columns(H), device="cuda")
    ep.ep_quantize_rows(x, q, s)
    ep.ep_quantize_rows(x[-n:], q2, s2)
    assert same(q[-n:], q2) and torch.equal(s[-n:], s2)
    # every token to its own expert row, last to first expert and back
    lid, size = ep.ep_register_layer(2, 1, H, T, 1)
    R, h = ep.ep_recv_capacity(lid), ep.alloc_handle(lid, size)
    idx = (torch.arange(T, device="cuda") % 2)[:, None].contiguous()
    ep.ep_prepare(h, idx, torch.empty(2, dtype=torch.int32, device="cuda"), 1)
    slots = torch.empty(T, 1, dtype=torch.int32, device="cuda")
    ep.ep_token_slots(h, slots)
    rq, rs, rw = torch.empty(R, H, dtype=F8, device="cuda"), torch.empty(R, columns(H), device="cuda"), torch.empty(R, device="cuda")
    ep.ep_dispatch_f8(h, idx, q, s, torch.ones(T, 1, device="cuda"), rq, rs, rw)
    at = slots[-n:, 0].long()
    assert int(at.max()) * H > 1 << 31
    assert same(rq.view(torch.uint8)[at], q2) and torch.equal(rs[at], s2)
    y, total = torch.empty_like(x), x.clone()
    ep.ep_rmsnorm(x, w, y=y, residual=total, sum=total, q=q, scales=s)
    y2, t2 = torch.empty_like(x[-n:]), torch.empty_like(x[-n:])
    ep.ep_rmsnorm(x[-n:], w, y=y2, residual=x[-n:], sum=t2, q=q2, scales=s2)
    assert torch.equal(y[-n:], y2) and torch.equal(total[-n:], t2) and same(q[-n:], q2) and torch.equal(s[-n:], s2)
    dw = torch.empty(H, device="cuda")
    ep.ep_rmsnorm_bwd(x, total, w, y, dw, ep.rmsnorm_bwd_workspace(T, H))
    ep.ep_rmsnorm_bwd(x[-n:], t2, w, y2, dw, ep.rmsnorm_bwd_workspace(n, H))
    assert torch.equal(y[-n:], y2)
