"""A whole Mixture-of-Experts layer on libep's calls: router, routing map,
dispatch, the experts' gated products, combine, and the backward pass; and the
same forward pass with 4-bit expert weights for serving.

    layer = MoELayer(experts=E, top_k=K, hidden=H, ffn=F, max_tokens=T)
    out = layer.forward(x, gate, w13, w2)          # training: keeps what backward reads
    grads = layer.backward(grad_out, w13, w2, gate)
    q = layer.quantize(w13, w2)                    # once, when weights are loaded
    out = layer.decode(x, gate, q)                 # serving, 4-bit weights

Weights: gate [E, H]; w13 [E, 2F, H] (gate rows, then up rows); w2 [E, H, F].
Every buffer is allocated once; a step's routing stays on the device, so
forward, backward and decode only enqueue work and can be captured in a CUDA
graph (the gate's small matrix products are torch's).

As a command it runs one layer and prints the time of a training step and of
a decode step:

    python -m combine_ep_prepare_gb300.moe_layer --tokens 4096 --experts 32 --top-k 4 --hidden 2048 --ffn 1024
"""
from __future__ import annotations

import argparse
from typing import NamedTuple, Optional

import torch

import combine_ep_prepare_gb300 as ep


class Grads(NamedTuple):
    x: torch.Tensor
    gate: torch.Tensor
    w13: torch.Tensor
    w2: torch.Tensor


class QuantizedExperts(NamedTuple):
    w13: torch.Tensor
    s13: torch.Tensor
    w2: torch.Tensor
    s2: torch.Tensor


class MoELayer:
    def __init__(self, experts: int, top_k: int, hidden: int, ffn: int, max_tokens: int, dtype=torch.bfloat16,
                 score: str = "softmax", normalize: bool = True, num_groups: int = 1, topk_groups: int = 1,
                 scale: float = 1.0, alignment: int = 1, grad_dtype=torch.float32, device="cuda"):
        self.experts, self.top_k, self.hidden, self.ffn = experts, top_k, hidden, ffn
        self.dtype, self.alignment, self.grad_dtype, self.device = dtype, alignment, grad_dtype, device
        self.routing = dict(score=score, normalize=normalize, num_groups=num_groups, topk_groups=topk_groups, scale=scale)
        lid, size = ep.ep_register_layer(experts, top_k, hidden, max_tokens, alignment, dtype=dtype)
        rows = ep.ep_recv_capacity(lid)
        self.handle = ep.alloc_handle(lid, size, device)
        new = lambda *shape, dtype=dtype: torch.empty(*shape, dtype=dtype, device=device)  # noqa: E731
        f32, i64 = torch.float32, torch.int64
        self.idx, self.weights = new(max_tokens, top_k, dtype=i64), new(max_tokens, top_k, dtype=f32)
        self.counts = new(experts, dtype=torch.int32)
        self.recv, self.recv_weights = new(rows, hidden), new(rows, dtype=f32)
        self.pre, self.act, self.expert_out = new(rows, 2 * ffn), new(rows, ffn), new(rows, hidden)
        # backward: gradients of the expert rows and of the receive rows, of pre and of the rows' weights
        self.d_rows, self.d_pre, self.d_weights = new(rows, hidden), new(rows, 2 * ffn), new(rows, dtype=f32)
        self.x: Optional[torch.Tensor] = None

    def _route(self, x, gate, bias):
        """Router, routing map and dispatch of a batch.  The buffers are then no
        longer those of an earlier forward."""
        T, self.x = x.shape[0], None
        self.logits = x.float() @ gate.float().t()
        self.t_idx, self.t_weights = self.idx[:T], self.weights[:T]
        ep.ep_router(self.logits, self.t_idx, self.t_weights, bias=bias, **self.routing)
        ep.ep_prepare(self.handle, self.t_idx, self.counts, self.alignment)
        ep.ep_dispatch(self.handle, self.t_idx, x, self.t_weights, self.recv, self.recv_weights)

    def forward(self, x, gate, w13, w2, bias=None) -> torch.Tensor:
        """x [T, H] -> [T, H]; keeps what backward reads until the next call."""
        self._route(x, gate, bias)
        ep.ep_expert_gemm_swiglu(self.handle, self.recv, w13, self.act, pre=self.pre)
        ep.ep_expert_gemm(self.handle, self.act, w2, self.expert_out)
        out = torch.empty_like(x)
        ep.ep_combine_weighted(self.handle, self.expert_out, self.recv_weights, out)
        self.x = x
        return out

    def backward(self, grad, w13, w2, gate, into: Optional[Grads] = None) -> Grads:
        """Gradients of the last forward from the gradient of its result.
        into: earlier gradients, whose w13 and w2 are added to."""
        h, T = self.handle, grad.shape[0]
        if self.x is None or self.x.shape[0] != T:
            raise ValueError("backward needs the batch of the last forward: %d rows given" % T)
        if into is None:
            dw13 = torch.empty(w13.shape, dtype=self.grad_dtype, device=self.device)
            dw2 = torch.empty(w2.shape, dtype=self.grad_dtype, device=self.device)
        else:
            dw13, dw2 = into.w13, into.w2
        add = into is not None
        ep.ep_combine_weighted_bwd(h, grad, self.expert_out, self.recv_weights, self.d_rows, self.d_weights)
        ep.ep_expert_wgrad(h, self.d_rows, self.act, dw2, accumulate=add)
        ep.ep_expert_dgrad_swiglu(h, self.d_rows, w2, self.pre, self.d_pre)
        ep.ep_expert_wgrad(h, self.d_pre, self.recv, dw13, accumulate=add)
        ep.ep_expert_dgrad(h, self.d_pre, w13, self.d_rows)
        dx, d_topk = torch.empty_like(self.x), torch.empty_like(self.t_weights)
        ep.ep_dispatch_bwd(h, self.d_rows, self.d_weights, dx, d_topk)
        d_logits = torch.empty_like(self.logits)
        ep.ep_router_bwd(self.logits, self.t_idx, d_topk, d_logits, score=self.routing["score"],
                         normalize=self.routing["normalize"], scale=self.routing["scale"])
        d_gate = d_logits.t() @ self.x.float()
        dx = (dx.float() + d_logits @ gate.float()).to(self.dtype)
        return Grads(dx, d_gate if into is None else into.gate + d_gate, dw13, dw2)

    def quantize(self, w13, w2, group: int = 128) -> QuantizedExperts:
        return QuantizedExperts(*ep.pack_w4(w13, group), *ep.pack_w4(w2, group))

    def decode(self, x, gate, q: QuantizedExperts, bias=None) -> torch.Tensor:
        """The forward pass with 4-bit expert weights; nothing is kept for a backward."""
        self._route(x, gate, bias)
        ep.ep_expert_gemv_w4_swiglu(self.handle, self.recv, q.w13, q.s13, self.act)
        ep.ep_expert_gemv_w4(self.handle, self.act, q.w2, q.s2, self.expert_out)
        out = torch.empty_like(x)
        ep.ep_combine_weighted(self.handle, self.expert_out, self.recv_weights, out)
        return out


def _time(step, n: int) -> float:
    """Milliseconds of one of n steps, after two untimed ones."""
    for _ in range(2):
        step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(n):
        step()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) / n


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description="One MoE layer: the time of a training step and of a 4-bit decode step.")
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--decode-tokens", type=int, default=16)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--ffn", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    bf16 = torch.bfloat16
    rand = lambda *shape, scale=1.0: (torch.randn(*shape, generator=g, device="cuda") * scale).to(bf16)  # noqa: E731
    gate = rand(a.experts, a.hidden, scale=a.hidden ** -0.5)
    w13 = rand(a.experts, 2 * a.ffn, a.hidden, scale=a.hidden ** -0.5)
    w2 = rand(a.experts, a.hidden, a.ffn, scale=a.ffn ** -0.5)
    x, grad = rand(a.tokens, a.hidden), rand(a.tokens, a.hidden)
    layer = MoELayer(a.experts, a.top_k, a.hidden, a.ffn, max(a.tokens, a.decode_tokens))

    def train():
        layer.forward(x, gate, w13, w2)
        layer.backward(grad, w13, w2, gate)

    ms = _time(train, a.steps)
    flops = 3 * 6 * a.tokens * a.top_k * a.hidden * a.ffn
    print("training step: %d tokens, %d experts, top %d, %d -> %d: %.3f ms, %.0f TFLOP/s in the expert products"
          % (a.tokens, a.experts, a.top_k, a.hidden, a.ffn, ms, flops / ms / 1e9))
    q = layer.quantize(w13, w2)
    few = x[:a.decode_tokens]
    ms = _time(lambda: layer.decode(few, gate, q), a.steps)
    print("decode step, 4-bit weights: %d tokens: %.3f ms" % (a.decode_tokens, ms))
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
