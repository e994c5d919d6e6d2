"""A few tokens' whole layer against the same layer in 64 bits, on the experts
that it chose (which are compared with the choice from 64-bit logits).

Tolerances.  A sum of n products in float32 is off by at most n 2^-23 of its
magnitudes.  16-bit weights round a to the payload type (2^-8, 2^-11).  8-bit
weights quantise a: a computed value within d of the exact one may land on any
e4m3 value that the interval [a - d, a + d] rounds to, so the interval's ends
are quantised too and the spread enters the bound (the block's scale moves by
d as well).  The result is rounded once.
"""
import pytest
import torch

from combine_ep_prepare_gb300 import workloads as wl
from tests.test_experts_gpu import ACT, STEP, UNIT, ep  # noqa: F401
from tests.test_f8_rows_gpu import quantize

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


class Few:
    def __init__(self, ep, E, K, H, F, T, dtype="bf16", f8=False, seed=60, **route):  # noqa: F811
        dt = wl.TORCH_PAYLOAD[dtype]
        new = lambda a, b, n, scale=1.0: (wl.payload_normal(a, b, seed + n, "fp32") * scale)  # noqa: E731
        self.E, self.K, self.H, self.F, self.T, self.dtype, self.f8, self.route = E, K, H, F, T, dtype, f8, route
        self.x = new(T, H, 1).to(dt).cuda()
        self.gate = new(E, H, 2, 1.5 * H ** -0.5).to(dt).cuda()
        self.w13 = new(E * 2 * F, H, 3, H ** -0.5).to(dt).view(E, 2 * F, H).cuda()
        self.w2 = new(E * H, F, 4, F ** -0.5).to(dt).view(E, H, F).cuda()
        self.s13 = self.s2 = None
        self.v13, self.v2 = self.w13, self.w2
        if f8:
            self.w13, self.s13 = ep.pack_f8(self.w13)
            self.w2, self.s2 = ep.pack_f8(self.w2)
            self.v13, self.v2 = (w.double() * s.double().repeat_interleave(128, 1)[:, :w.shape[1]].repeat_interleave(128, 2)[:, :, :w.shape[2]]
                                 for w, s in ((self.w13, self.s13), (self.w2, self.s2)))
        self.work = ep.moe_few_workspace(E, K, H, F, T)
        self.out = torch.full((T, H), float("nan"), dtype=dt, device="cuda")
        self.idx = torch.full((T, K), -7, dtype=torch.int64, device="cuda")
        self.p = torch.full((T, K), float("nan"), device="cuda")

    def run(self, ep, **kw):  # noqa: F811
        ep.ep_moe_few(self.x, self.gate, self.w13, self.w2, self.out, self.idx, self.p, self.work, s13=self.s13, s2=self.s2,
                      **{**self.route, **kw})
        return self.out

    def check(self, bias=None):
        x, dt = self.x.double(), self.dtype
        z = x @ self.gate.double().t()
        score = self.route.get("score", "softmax")
        sg = torch.sigmoid(z)
        idx = self.idx.clamp_min(0)
        live = self.idx >= 0
        if self.route.get("num_groups", 1) == 1:
            v = z if score == "softmax" else sg if bias is None else sg + bias.double()
            n = torch.isfinite(v).sum(1).clamp_max(self.K)
            want = torch.topk(v, self.K, dim=1).indices
            keep = torch.arange(self.K, device="cuda")[None] < n[:, None]
            assert torch.equal(torch.where(keep, want, -1), self.idx)
        if score == "softmax":
            p = torch.softmax(z.gather(1, idx).masked_fill(~live, -torch.inf), 1) if self.route.get("normalize", True) else torch.softmax(z, 1).gather(1, idx)
        else:
            p = sg.gather(1, idx) * live
            p = p / p.sum(1, keepdim=True).clamp_min(1e-300) if self.route.get("normalize", True) else p
        p = torch.nan_to_num(p) * live * self.route.get("scale", 1.0)
        assert bool(((self.p.double() - p).abs() <= 1e-5 * p + 1e-30).all())
        p = self.p.double()
        xv = x
        if self.f8:
            q, s = quantize(self.x)
            xv = (q.double() * s.double().repeat_interleave(128, 1)[:, :self.H]).cuda()
        want, bound = torch.zeros_like(x), torch.zeros_like(x)
        n1, n2 = ((128 + self.H // 128 + 4) * STEP, (128 + self.F // 128 + 4) * STEP) if self.f8 else (self.H * STEP, self.F * STEP)
        for e in torch.unique(self.idx[live]).tolist():
            t, k = (self.idx == e).nonzero(as_tuple=True)
            w13, w2 = self.v13[e].double(), self.v2[e].double()
            g, u = (xv[t] @ w13.t()).chunk(2, dim=1)
            dg, du = (n1 * (xv[t].abs() @ w13.abs().t())).chunk(2, dim=1)
            sgm = torch.sigmoid(g)
            a = g * sgm * u
            off = 1.1 * dg * (u.abs() + du) + (g * sgm).abs() * du + ACT * (1 + g.abs()) * a.abs()
            if self.f8:
                m = a.abs().view(len(t), -1, 128).amax(2).clamp_min(2.0 ** -100)
                dm = off.view(len(t), -1, 128).amax(2) / m
                wide = lambda b: b.repeat_interleave(128, 1)  # noqa: E731
                v, dv = a / wide(m) * 448, (off + a.abs() * (wide(dm) + 4 * STEP)) / wide(m) * 448
                f = lambda y: y.clamp(-448, 448).float().to(F8).double()  # noqa: E731
                centre = f(v)
                spread = (f(v + dv) - f(v - dv)).abs()
                av, off = centre * wide(m) / 448, (spread + centre.abs() * (wide(dm) + 4 * STEP)) * wide(m) / 448
            else:
                av, off = a, off + UNIT[dt] * (a.abs() + off) + 2.0 ** -25
            y = av @ w2.t()
            by = off @ w2.abs().t() + n2 * ((av.abs() + off) @ w2.abs().t())
            want.index_add_(0, t, y * p[t, k][:, None])
            bound.index_add_(0, t, (by + 2 * self.K * STEP * (av.abs() @ w2.abs().t())) * p[t, k].abs()[:, None])
        d = (self.out.double() - want).abs()
        bound = bound + UNIT[dt] * (want.abs() + bound) + 2.0 ** -25
        assert bool(torch.isfinite(self.out).all())
        assert bool((d <= bound).all()), (d / bound).max().item()


SHAPES = [(1, 1, 8, 8, 1), (4, 2, 64, 24, 3), (8, 2, 256, 128, 8), (16, 4, 520, 136, 9), (128, 8, 1024, 256, 16),
          (6, 6, 328, 1032, 17), (3, 2, 2048, 64, 31), (40, 5, 136, 200, 32), (1024, 32, 64, 8, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_16_bit_weights(ep, shape, dtype):  # noqa: F811
    m = Few(ep, *shape, dtype=dtype)
    m.run(ep)
    m.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", [(1, 1, 16, 128, 1), (4, 2, 64, 128, 3), (8, 2, 256, 256, 8), (16, 4, 528, 384, 9), (128, 8, 1024, 256, 16),
                                   (6, 6, 336, 1152, 17), (3, 2, 2048, 128, 31), (40, 5, 144, 256, 32)], ids=str)
def test_8_bit_weights(ep, shape, dtype):  # noqa: F811
    m = Few(ep, *shape, dtype=dtype, f8=True)
    m.run(ep)
    m.check()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("route", [dict(score="sigmoid"), dict(score="sigmoid", normalize=False, scale=2.5), dict(normalize=False),
                                   dict(score="sigmoid", num_groups=4, topk_groups=2), dict(num_groups=8, topk_groups=3)], ids=str)
def test_routing(ep, route, f8):  # noqa: F811
    m = Few(ep, 32, 4, 256, 128, 13, f8=f8, **route)
    m.run(ep)
    m.check()
    logits = (m.x.double() @ m.gate.double().t()).float()
    idx, p = torch.empty_like(m.idx), torch.empty_like(m.p)
    ep.ep_router(logits, idx, p, **route)
    assert torch.equal(idx, m.idx)


def test_selection_bias_and_float32_gate(ep):  # noqa: F811
    m = Few(ep, 32, 4, 256, 128, 7, score="sigmoid")
    bias = (wl.payload_normal(1, 32, 70, "fp32")[0] * 0.3).cuda()
    m.gate = m.gate.float()
    m.run(ep, bias=bias)
    m.check(bias=bias)


def test_infinite_logits_are_never_chosen(ep):  # noqa: F811
    """A token with -inf for most experts gets fewer choices; one with none gets zeros."""
    m = Few(ep, 8, 3, 64, 64, 4)
    m.x.zero_()
    m.x[:, 0] = torch.tensor([1.0, 1.0, 0.0, 1.0])
    m.x[1, 1:9] = 1
    m.gate.zero_()
    m.gate[:6, 0] = -torch.inf
    m.x[2, 1:9] = torch.tensor([1.0, 2, 3, 4, 5, 6, 7, 8])
    m.gate[:, 1:9] = torch.eye(8) * 0.5
    m.run(ep)
    # 0 * -inf is NaN, never chosen: token 2 has two choices like the others
    assert torch.equal((m.idx >= 0).sum(1).cpu(), torch.tensor([2, 2, 2, 2])) and bool((m.p[m.idx < 0] == 0).all())
    assert bool(torch.isfinite(m.out).all())
    m.gate[:, 0] = -torch.inf
    m.run(ep)
    assert bool((m.idx == -1).all()) and bool((m.p == 0).all()) and bool((m.out == 0).all())


def test_same_token_twice_and_again(ep):  # noqa: F811
    """Equal tokens get equal rows, and a second call the same bits, whatever the workspace holds."""
    for f8 in (False, True):
        m = Few(ep, 16, 4, 512, 256, 12, f8=f8)
        m.x[7] = m.x[2]
        m.run(ep)
        first = m.out.clone()
        assert torch.equal(m.out[7], m.out[2])
        m.work.fill_(0xff)
        m.run(ep)
        assert torch.equal(m.out, first)
        assert int(m.work[:4].view(torch.int32)) == 0


def test_no_tokens(ep):  # noqa: F811
    m = Few(ep, 4, 2, 64, 64, 1)
    before = ep.ep_launch_count()
    ep.ep_moe_few(m.x[:0], m.gate, m.w13, m.w2, m.out[:0], m.idx[:0], m.p[:0], m.work)
    assert ep.ep_launch_count() == before


@pytest.mark.parametrize("f8", [False, True])
def test_captured_and_on_another_stream(ep, f8):  # noqa: F811
    m = Few(ep, 16, 4, 512, 256, 5, f8=f8)
    m.run(ep)
    first, x = m.out.clone(), m.x.clone()
    m.run(ep)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=other):
        m.run(ep)
        m.run(ep)
    for n in range(4):
        m.x.copy_(x.roll(n, 0))
        m.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(m.out, first.roll(n, 0))


def test_agrees_with_the_8_bit_path(ep):  # noqa: F811
    """The same tokens over quantise, dispatch, the 8-bit products and the weighted combine."""
    E, K, H, F, T = 16, 4, 512, 256, 24
    m = Few(ep, E, K, H, F, T, f8=True)
    m.run(ep)
    m.check()
    lid, size = ep.ep_register_layer(E, K, H, T, 1)
    R, h = ep.ep_recv_capacity(lid), ep.alloc_handle(lid, size)
    ep.ep_prepare(h, m.idx, torch.empty(E, dtype=torch.int32, device="cuda"), 1)
    f8 = lambda n, w: (torch.empty(n, w, dtype=F8, device="cuda"), torch.empty(n, ep.scale_columns(w), device="cuda"))  # noqa: E731
    (q, s), (rq, rs), (aq, asc) = f8(T, H), f8(R, H), f8(R, F)
    rw, y, out = torch.empty(R, device="cuda"), torch.empty(R, H, dtype=m.x.dtype, device="cuda"), torch.empty_like(m.out)
    ep.ep_quantize_rows(m.x, q, s)
    ep.ep_dispatch_f8(h, m.idx, q, s, m.p, rq, rs, rw)
    ep.ep_expert_gemm_f8_swiglu(h, rq, rs, m.w13, m.s13, act_q=aq, act_scales=asc)
    ep.ep_expert_gemm_f8(h, aq, asc, m.w2, m.s2, y)
    ep.ep_combine_weighted(h, y, rw, out)
    # K expert outputs rounded to bf16 and the sum once more; a value of act on a border may land one e4m3 step away
    assert ((out.double() - m.out.double()).norm() / m.out.double().norm()).item() <= (K ** 0.5 + 1) * 2.0 ** -8


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("H,F", [(32768, 128), (128, 32768)])
def test_longest_rows(ep, H, F, f8):  # noqa: F811
    m = Few(ep, 3, 2, H, F, 32, f8=f8)
    m.run(ep)
    m.check()


@pytest.mark.parametrize("f8", [False, True])
def test_nan_tokens_stay_alone(ep, f8):  # noqa: F811
    """No logit of a token with a NaN can be chosen: it gets zeros, the others their own results."""
    m = Few(ep, 16, 4, 512, 256, 11, f8=f8)
    m.x[3, 17] = float("nan")
    m.run(ep)
    assert bool((m.idx[3] == -1).all()) and bool((m.out[3] == 0).all())
    m.x[3] = 0  # of no weight in what the others are compared with
    keep = m.idx.clone()
    want = Few(ep, 16, 4, 512, 256, 11, f8=f8)
    want.x, want.out, want.idx, want.p = (t[torch.arange(11) != 3] for t in (m.x, m.out, keep, m.p))
    want.check()


def test_two_graphs_on_one_workspace_and_two_streams(ep):  # noqa: F811
    """Two captured calls of other sizes take turns on one workspace; with a workspace each they may run at once."""
    a, b = Few(ep, 64, 8, 1024, 256, 16, f8=True), Few(ep, 16, 4, 512, 256, 5, seed=90)
    want = [m.run(ep).clone() for m in (a, b)]
    both = torch.empty(max(a.work.numel(), b.work.numel()), dtype=torch.uint8, device="cuda")
    own = [a.work, b.work]
    a.work = b.work = both
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, m in zip(graphs, (a, b)):
        with torch.cuda.graph(g):
            m.run(ep)
    for n in (0, 1, 1, 0, 1, 0, 0):
        for m in (a, b):
            m.out.fill_(float("nan"))
        graphs[n].replay()
        assert torch.equal((a, b)[n].out, want[n])
    a.work, b.work = own
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s, m in zip(streams, (a, b)):
            m.run(ep, stream=s)
    torch.cuda.synchronize()
    for m, w in zip((a, b), want):
        assert int(m.work[:4].view(torch.int32)) == 0 and torch.equal(m.out, w)
