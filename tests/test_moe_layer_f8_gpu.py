"""The layer of moe_layer.py with 8-bit rows and weights, and of a few tokens,
against the same layer in float64 autograd on the layer's own choice of experts
and the values that its 8-bit weights stand for.

Tolerances are on norms (of the difference over the result's).  A value rounded
to e4m3 is off by at most 2^-4 of itself.  The forward pass rounds the rows
twice (its input and act): 2 * 2^-4.  A gradient depends on those and on the two
roundings of rows' gradients: 4 * 2^-4, with ten roundings of 2^-8 beside them.
"""
import pytest
import torch

from tests.test_moe_layer_gpu import REL, moe, off, problem, reference  # noqa: F401

pytestmark = pytest.mark.gpu
Q = 2.0 ** -4


def values(w, s):
    n, k = w.shape[1:]
    return w.double() * s.double().repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E,K,H,F,T,kw", [
    (8, 2, 64, 128, 100, dict(score="softmax")), (16, 4, 272, 256, 33, dict(score="sigmoid", num_groups=4, topk_groups=2, scale=2.5)),
    (4, 1, 256, 128, 300, dict(score="softmax", normalize=False, alignment=128)), (6, 3, 144, 128, 1, dict(score="sigmoid", normalize=False))])
def test_forward_and_gradients(moe, E, K, H, F, T, kw, dtype):  # noqa: F811
    x, gate, w13, w2, grad = problem(E, K, H, F, T, dtype)
    layer = moe.MoELayer(E, K, H, F, T + 5, dtype=dtype, **kw)
    q = layer.quantize_f8(w13, w2)
    out = layer.forward_f8(x, gate, q)
    grads = layer.backward_f8(grad, q, gate)
    leaves = [x.double().requires_grad_(), gate.double().requires_grad_(), values(q.w13, q.s13).requires_grad_(), values(q.w2, q.s2).requires_grad_()]
    want = reference(*leaves, layer.t_idx, kw["score"], kw.get("normalize", True), kw.get("scale", 1.0))
    assert off(out, want) <= 2 * Q + REL[dtype]
    for name, got, ref in zip(grads._fields, grads, torch.autograd.grad(want, leaves, grad.double())):
        assert off(got, ref) <= 4 * Q + REL[dtype], name


def test_norm_residual_and_what_comes_down_the_stream(moe):  # noqa: F811
    E, K, H, F, T, eps = 8, 2, 256, 128, 77, 1e-5
    x, gate, w13, w2, grad = problem(E, K, H, F, T, torch.bfloat16)
    res, down = problem(E, K, H, F, T, torch.bfloat16, seed=2)[0], problem(E, K, H, F, T, torch.bfloat16, seed=3)[0]
    w = (1 + 0.2 * problem(1, 1, H, 8, 1, torch.bfloat16, seed=4)[0][0]).to(torch.bfloat16)
    layer = moe.MoELayer(E, K, H, F, T)
    q = layer.quantize_f8(w13, w2)
    out, total = layer.forward_f8(x, gate, q, norm=w, residual=res, eps=eps)
    assert torch.equal(total, (x.float() + res.float()).to(torch.bfloat16))
    grads = layer.backward_f8(grad, q, gate, grad_sum=down)
    h, ww, g = total.double().requires_grad_(), w.double().requires_grad_(), gate.double().requires_grad_()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * ww
    want = reference(y, g, values(q.w13, q.s13), values(q.w2, q.s2), layer.t_idx, "softmax", True, 1.0)
    assert off(out, want) <= 2 * Q + REL[torch.bfloat16]
    dh, dw, dg = torch.autograd.grad(want, (h, ww, g), grad.double())
    assert off(grads.x, dh + down.double()) <= 4 * Q + REL[torch.bfloat16]
    assert off(grads.norm, dw) <= 4 * Q + REL[torch.bfloat16] and off(grads.gate, dg) <= 4 * Q + REL[torch.bfloat16]


def test_backward_f8_follows_its_forward_alone(moe):  # noqa: F811
    E, K, H, F, T = 4, 2, 64, 128, 10
    x, gate, w13, w2, grad = problem(E, K, H, F, T, torch.bfloat16)
    layer = moe.MoELayer(E, K, H, F, T)
    q = layer.quantize_f8(w13, w2)
    with pytest.raises(ValueError, match="last forward_f8"):
        layer.backward_f8(grad, q, gate)
    layer.forward_f8(x, gate, q)
    with pytest.raises(ValueError, match="last forward:"):
        layer.backward(grad, w13, w2, gate)
    with pytest.raises(ValueError, match="grad_sum"):
        layer.backward_f8(grad, q, gate, grad_sum=grad)
    layer.forward(x, gate, w13, w2)
    with pytest.raises(ValueError, match="last forward_f8"):
        layer.backward_f8(grad, q, gate)
    layer.forward_f8(x, gate, q)
    first = layer.backward_f8(grad, q, gate)
    layer.few(x, gate, w13, w2)  # uses none of their buffers
    assert all(torch.equal(a, b) for a, b in zip(first[:4], layer.backward_f8(grad, q, gate)[:4]))
    with pytest.raises(Exception):
        layer.forward_f8(x, gate, q._replace(s13=q.s13[:, :1].contiguous()))
    with pytest.raises(ValueError, match="last forward_f8"):
        layer.backward_f8(grad, q, gate)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 7, 32])
def test_few(moe, T, dtype):  # noqa: F811
    E, K, H, F = 8, 2, 256, 128
    x, gate, w13, w2, _ = problem(E, K, H, F, T, dtype)
    layer = moe.MoELayer(E, K, H, F, T, dtype=dtype)
    q = layer.quantize_f8(w13, w2)
    out = layer.few(x, gate, w13, w2)
    assert off(out, reference(x.double(), gate.double(), w13.double(), w2.double(), layer.few_idx, "softmax", True, 1.0)) <= REL[dtype]
    out = layer.few(x, gate, q)
    want = reference(x.double(), gate.double(), values(q.w13, q.s13), values(q.w2, q.s2), layer.few_idx, "softmax", True, 1.0)
    assert off(out, want) <= 2 * Q + REL[dtype]
    # the same tokens over the batched 8-bit path choose and quantise alike
    assert off(layer.forward_f8(x, gate, q), out.double()) <= (K ** 0.5 + 1) * 2.0 ** -8
    assert torch.equal(layer.t_idx, layer.few_idx)


def test_step_captured_in_a_graph(moe):  # noqa: F811
    E, K, H, F, T = 8, 2, 128, 128, 20
    x, gate, w13, w2, grad = problem(E, K, H, F, T, torch.bfloat16)
    norm = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    layer = moe.MoELayer(E, K, H, F, T)
    q = layer.quantize_f8(w13, w2)

    def step():
        out = layer.forward_f8(x, gate, q, norm=norm, residual=grad)
        return (*out, *layer.backward_f8(grad, q, gate), layer.few(x, gate, q), layer.few(x, gate, w13, w2))

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


def test_command_times_the_8_bit_step_and_few(moe, capsys):  # noqa: F811
    assert moe.main(["--tokens", "64", "--experts", "8", "--top-k", "2", "--hidden", "256", "--ffn", "128", "--steps", "2"]) == 0
    said = capsys.readouterr().out
    assert "8-bit rows and weights" in said and said.count("two kernels") == 2
