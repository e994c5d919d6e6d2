"""The whole layer of moe_layer.py against the same layer in float64 autograd,
on the layer's own choice of experts.

Tolerances are on norms (of the difference over the result's).  fp32: four
products deep, each sum of n <= 256 terms off by at most n 2^-24, so 4 * 256 *
2^-24 < 6.2e-5.  16-bit types: at most ten roundings of 2^-8 (bf16) or 2^-11
(fp16) each between inputs and result.  4-bit: the same against the dequantised
weights.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

REL = {torch.float32: 4 * 256 * 2.0 ** -24, torch.bfloat16: 10 * 2.0 ** -8, torch.float16: 10 * 2.0 ** -11}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_ep_prepare_gb300 import moe_layer
    return moe_layer


def off(got, want):
    return ((got.double() - want).norm() / want.norm().clamp_min(1e-30)).item()


def problem(E, K, H, F, T, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dtype).cuda()  # noqa: E731
    return (r(T, H), r(E, H, scale=H ** -0.5), r(E, 2 * F, H, scale=H ** -0.5), r(E, H, F, scale=F ** -0.5), r(T, H))


def reference(x, gate, w13, w2, idx, score, normalize, scale):
    logits = x @ gate.t()
    if score == "sigmoid":
        w = torch.sigmoid(logits).gather(1, idx)
        w = w / w.sum(1, keepdim=True) if normalize else w
    else:
        w = torch.softmax(logits.gather(1, idx), 1) if normalize else torch.softmax(logits, 1).gather(1, idx)
    out = torch.zeros_like(x)
    for k in range(idx.shape[1]):
        for e in range(gate.shape[0]):
            t = (idx[:, k] == e).nonzero()[:, 0]
            if t.numel():
                g, u = (x[t] @ w13[e].t()).chunk(2, dim=1)
                out = out.index_add(0, t, (torch.nn.functional.silu(g) * u @ w2[e].t()) * (w[t, k] * scale)[:, None])
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E,K,H,F,T,kw", [
    (8, 2, 64, 40, 100, dict(score="softmax")), (16, 4, 128, 72, 33, dict(score="sigmoid", num_groups=4, topk_groups=2, scale=2.5)),
    (4, 1, 256, 128, 300, dict(score="softmax", normalize=False, alignment=128)), (6, 3, 72, 64, 1, dict(score="sigmoid", normalize=False))])
def test_layer_forward_and_gradients(moe, E, K, H, F, T, kw, dtype):
    x, gate, w13, w2, grad = problem(E, K, H, F, T, dtype)
    layer = moe.MoELayer(E, K, H, F, T + 5, dtype=dtype, **kw)
    out = layer.forward(x, gate, w13, w2)
    grads = layer.backward(grad, w13, w2, gate)
    leaves = [t.double().requires_grad_() for t in (x, gate, w13, w2)]
    want = reference(*leaves, layer.t_idx, kw["score"], kw.get("normalize", True), kw.get("scale", 1.0))
    assert off(out, want) <= REL[dtype]
    dx, dgate, dw13, dw2 = torch.autograd.grad(want, leaves, grad.double())
    for name, got, ref in (("x", grads.x, dx), ("gate", grads.gate, dgate), ("w13", grads.w13, dw13), ("w2", grads.w2, dw2)):
        assert off(got, ref) <= REL[dtype], name
    # accumulated onto the first: twice the gradients
    first13, first2 = grads.w13.clone(), grads.w2.clone()
    layer.forward(x, gate, w13, w2)
    twice = layer.backward(grad, w13, w2, gate, into=grads)
    assert torch.equal(twice.w13, 2 * first13) and torch.equal(twice.w2, 2 * first2)


def test_backward_without_forward_is_refused(moe):
    x, gate, w13, w2, grad = problem(4, 2, 64, 64, 10, torch.bfloat16)
    layer = moe.MoELayer(4, 2, 64, 64, 16)
    with pytest.raises(ValueError, match="last forward"):
        layer.backward(grad, w13, w2, gate)
    layer.forward(x[:5], gate, w13, w2)
    with pytest.raises(ValueError, match="last forward"):
        layer.backward(grad, w13, w2, gate)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 7, 40])
def test_decode_with_4_bit_weights(moe, T, dtype):
    E, K, H, F, group = 8, 2, 256, 128, 64
    x, gate, w13, w2, _ = problem(E, K, H, F, T, dtype)
    layer = moe.MoELayer(E, K, H, F, T, dtype=dtype)
    q = layer.quantize(w13, w2, group)
    out = layer.decode(x, gate, q)

    def back(wq, s):
        v = torch.stack([wq & 15, wq >> 4], dim=3).flatten(2).double() - 8
        return v * s.double().repeat_interleave(group, dim=2)

    want = reference(x.double(), gate.double(), back(q.w13, q.s13), back(q.w2, q.s2), layer.t_idx, "softmax", True, 1.0)
    assert off(out, want) <= REL[dtype]


def test_step_captured_in_a_graph(moe):
    E, K, H, F, T = 8, 2, 128, 64, 50
    x, gate, w13, w2, grad = problem(E, K, H, F, T, torch.bfloat16)
    layer = moe.MoELayer(E, K, H, F, T)
    q = layer.quantize(w13, w2, 32)

    def step():
        out = layer.forward(x, gate, w13, w2)
        grads = layer.backward(grad, w13, w2, gate)
        return (out, *grads, layer.decode(x, gate, q))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (2, 3):
        x.copy_(problem(E, K, H, F, T, torch.bfloat16, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in captured]
        assert all(torch.equal(a, b) for a, b in zip(replayed, step()))


def test_command(moe, capsys):
    assert moe.main(["--tokens", "64", "--experts", "8", "--top-k", "2", "--hidden", "256", "--ffn", "128", "--steps", "2"]) == 0
    said = capsys.readouterr().out
    assert "training step" in said and "decode step" in said
