"""The layer with 8-bit rows and weights against the same arithmetic in float64
with the layer's own roundings in their places: 8-bit rows, activation and
gradients, and everything that passes through a 16-bit buffer.

Tolerances, on norms.  What remains between the two is the last rounding of a
result to its type (2^-8 or 2^-11 of each value, once; the gate's and the
weights' gradients are float32), and values that a sum's order moves across a
border.  Sums of at most 512 products are off by some 133 2^-23 of their
magnitudes (test_f8_products_gpu.py), so a share of 133 2^-23 / 2^-3 of the
values at most lands a step of e4m3 (2^-3) away, 2^-3 times the share's root in
norm, and four roundings to e4m3 lie on the longest way: FLIPS = 5.7e-3.  In 16
bits a share of 133 2^-23 / u goes a step u away: (133 2^-23 u)^(1/2), 3.5e-4 for
bf16 and less for fp16, for each of the six such roundings on that way.
"""
import pytest
import torch

from tests.test_f8_rows_gpu import quantize
from tests.test_moe_layer_f8_gpu import values
from tests.test_moe_layer_gpu import moe, off, problem  # noqa: F401

pytestmark = pytest.mark.gpu

SUM = 133 * 2.0 ** -23
FLIPS = 4 * 2.0 ** -3 * (SUM / 2.0 ** -3) ** 0.5
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def float32_bound(dtype):
    return FLIPS + 6 * (SUM * 2 * UNIT[dtype]) ** 0.5


def bound(dtype):
    return UNIT[dtype] + float32_bound(dtype)


def eight(x):
    """The values that rows quantised from x (rounded to float32) stand for."""
    q, s = quantize(x.float())
    return (q.double() * s.double().repeat_interleave(128, 1)[:, :x.shape[1]]).to(x.device)


def shares(logits, idx, kw):
    if kw["score"] == "sigmoid":
        w = torch.sigmoid(logits).gather(1, idx)
        w = w / w.sum(1, keepdim=True) if kw.get("normalize", True) else w
    else:
        w = torch.softmax(logits.gather(1, idx), 1) if kw.get("normalize", True) else torch.softmax(logits, 1).gather(1, idx)
    return w * kw.get("scale", 1.0)


def arithmetic(dtype, x, x8, gate, q, grad, idx, kw):
    """Result and gradients of the layer from its rows x (payload type, float64)
    and the 8-bit rows' values x8: (out, dx without the router's term, that
    term, dgate, dw13, dw2)."""
    r16 = lambda t: t.to(dtype).double()  # noqa: E731
    w13, w2 = values(q.w13, q.s13), values(q.w2, q.s2)
    logits = (x @ gate.t()).requires_grad_()
    p = shares(logits, idx, kw)
    ps = p.detach().float().double()
    out, dx, d_p = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(ps)
    dw13, dw2 = torch.zeros_like(w13), torch.zeros_like(w2)
    for k in range(idx.shape[1]):
        for e in range(gate.shape[0]):
            t = (idx[:, k] == e).nonzero()[:, 0]
            if not t.numel():
                continue
            pre = x8[t] @ w13[e].t()
            g, u = pre.chunk(2, 1)
            act = torch.nn.functional.silu(g) * u
            y = r16(eight(act) @ w2[e].t())
            out[t] += ps[t, k, None] * y
            d_p[t, k] = (grad[t] * y).sum(1)
            d_rows = r16(ps[t, k, None] * grad[t])
            dw2[e] += d_rows.t() @ r16(act)
            d_act = eight(d_rows) @ w2[e]
            g, u = r16(pre).chunk(2, 1)
            sg = torch.sigmoid(g)
            d_pre = r16(torch.cat([d_act * u * sg * (1 + g * (1 - sg)), d_act * g * sg], 1))
            dw13[e] += d_pre.t() @ x[t]
            dx[t] += r16(eight(d_pre) @ w13[e])
    d_logits, = torch.autograd.grad(p, logits, d_p)
    return out, r16(dx), d_logits @ gate, d_logits.t() @ x, dw13, dw2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E,K,H,F,T,kw", [
    (8, 2, 64, 128, 100, dict(score="softmax")), (16, 4, 272, 256, 33, dict(score="sigmoid", num_groups=4, topk_groups=2, scale=2.5)),
    (4, 1, 256, 128, 300, dict(score="softmax", normalize=False, alignment=128)), (6, 3, 144, 128, 1, dict(score="sigmoid", normalize=False))])
def test_forward_and_gradients(moe, E, K, H, F, T, kw, dtype):  # noqa: F811
    x, gate, w13, w2, grad = problem(E, K, H, F, T, dtype)
    layer = moe.MoELayer(E, K, H, F, T + 5, dtype=dtype, **kw)
    q = layer.quantize_f8(w13, w2)
    out = layer.forward_f8(x, gate, q)
    got = layer.backward_f8(grad, q, gate)
    want, dx, term, d_gate, d_w13, d_w2 = arithmetic(dtype, x.double(), eight(x), gate.double(), q, grad.double(), layer.t_idx, kw)
    assert off(out, want) <= bound(dtype)
    assert off(got.x, dx + term) <= bound(dtype)
    assert off(got.w13, d_w13) <= float32_bound(dtype) and off(got.w2, d_w2) <= float32_bound(dtype)
    assert off(got.gate, d_gate) <= float32_bound(dtype)
    assert off(dx, dx + term) > 5 * bound(dtype)  # a layer that lost the router's term would not have passed


def test_norm_residual_and_what_comes_down_the_stream(moe):  # noqa: F811
    E, K, H, F, T, eps, dtype = 8, 2, 256, 128, 77, 1e-5, torch.bfloat16
    x, gate, w13, w2, grad = problem(E, K, H, F, T, dtype)
    res, down = problem(E, K, H, F, T, dtype, seed=2)[0], problem(E, K, H, F, T, dtype, seed=3)[0]
    w = (1 + 0.2 * problem(1, 1, H, 8, 1, dtype, seed=4)[0][0]).to(dtype)
    layer = moe.MoELayer(E, K, H, F, T)
    q = layer.quantize_f8(w13, w2)
    out, total = layer.forward_f8(x, gate, q, norm=w, residual=res, eps=eps)
    got = layer.backward_f8(grad, q, gate, grad_sum=down)
    h, ww = total.double().requires_grad_(), w.double().requires_grad_()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * ww
    rows = y.detach().to(dtype).double()
    want, dx, term, d_gate, _, _ = arithmetic(dtype, rows, eight(y.detach()), gate.double(), q, grad.double(), layer.t_idx, dict(score="softmax"))
    assert off(out, want) <= bound(dtype) and off(got.gate, d_gate) <= float32_bound(dtype)
    dh, dw = torch.autograd.grad(y, (h, ww), (dx + term).to(dtype).double())
    # dh alone: the sum with what came down is rounded once
    left = (got.x.double() - down.double() - dh).norm()
    assert left <= float32_bound(dtype) * dh.norm() + UNIT[dtype] * (dh + down.double()).norm()
    assert off(got.norm, dw) <= float32_bound(dtype)
