"""An MoE layer on W ranks, forward and backward, from the framework's calls.

    python examples/moe_layer.py [--tokens 1024] [--hidden 7168] [--inner 2048] ...

Each rank has its tokens x [T, H]; rank p holds the experts [p K, (p + 1) K).
A token goes to its topk experts and gets the weighted sum of what they answer:

    y = x + sum_j weight_j * (silu(x Wg^T) * (x Wu^T)) Wd^T        (expert j's weights)

Forward: route, dispatch, expert_matmul (gated), expert_matmul,
combine_weighted.  Backward: combine_weighted_backward, both products'
gradients, combine_weighted without weights (the dispatch's gradient) and
route_backward.  No call waits for the device; ``status`` is read once a step.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import variable_size_all_gb300 as a2av  # noqa: E402


class MoeLayer:
    """Weights, buffers and the two passes.  ``capacity``: rows a rank can
    receive (a dispatch of more is refused on the device)."""

    def __init__(self, W, tokens, hidden, inner, experts, topk, dtype=torch.bfloat16,
                 capacity=None, score="softmax"):
        self.W, self.T, self.H, self.N, self.k = W, tokens, hidden, inner, topk
        self.E, self.K, self.dtype, self.score = experts, experts // W, dtype, score
        self.capacity = C = capacity or W * tokens * topk
        self.engine = a2av.A2av(W, out_capacity_rows=C)
        new = lambda *shape, dtype=dtype: [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(W)]
        K, T, H, N, k = self.K, tokens, hidden, inner, topk
        self.gate = torch.randn(experts, H, device="cuda") * H ** -0.5
        self.up = [(torch.randn(K, 2 * N, H, device="cuda") * H ** -0.5).to(dtype) for _ in range(W)]
        self.down = [(torch.randn(K, H, N, device="cuda") * N ** -0.5).to(dtype) for _ in range(W)]
        # what the forward pass fills and the backward pass reads
        self.keys, self.weights = new(T, k, dtype=torch.int32), new(T, k, dtype=torch.float32)
        self.counts = torch.empty(W, experts, dtype=torch.int64, device="cuda")
        self.splits = torch.empty(W, W, dtype=torch.int64, device="cuda")
        self.offsets = torch.empty(W, 2, W, dtype=torch.int64, device="cuda")
        self.pos = new(T * k, dtype=torch.int64)
        self.source = [torch.arange(T, dtype=torch.int32, device="cuda").repeat_interleave(k)
                       for _ in range(W)]
        self.received, self.pre = new(C, H), new(C, 2 * N)
        self.inner, self.answer, self.out = new(C, N), new(C, H), new(T, H)
        # gradients
        self.d_answer, self.d_inner, self.d_received = new(C, H), new(C, N), new(C, H)
        self.d_up, self.d_down = new(K, 2 * N, H), new(K, H, N)
        self.d_weights, self.d_x = new(T, k, dtype=torch.float32), new(T, H)

    def forward(self, x):
        e, K = self.engine, self.K
        self.x = x
        # the gate's product is a small dense one
        self.logits = [t.float() @ self.gate.T for t in x]
        e.route(self.logits, self.keys, self.weights, self.k, counts=self.counts, score=self.score)
        e.dispatch([t.view(torch.uint8) for t in x], self.source, [t.view(-1) for t in self.keys], K,
                   self.received, self.offsets, self.pos, self.H * x[0].element_size(),
                   in_splits=self.splits)
        e.expert_matmul(self.received, self.counts, self.up, self.inner, activation="silu", gated=True,
                        pre=self.pre)
        e.expert_matmul(self.inner, self.counts, self.down, self.answer)
        e.combine_weighted(self.answer, self.splits, self.keys, self.pos, K, self.weights, self.out,
                           residual=x)
        return self.out

    def backward(self, dy):
        """Gradients of x (returned), up, down and gate (kept in d_*)."""
        e, K = self.engine, self.K
        e.combine_weighted_backward(self.answer, self.splits, self.keys, self.pos, K, self.weights, dy,
                                    self.d_answer, self.d_weights)
        e.expert_matmul_backward(self.inner, self.counts, self.down, self.d_answer,
                                 d_rows=self.d_inner, d_weights=self.d_down)
        e.expert_matmul_backward(self.received, self.counts, self.up, self.d_inner,
                                 d_rows=self.d_received, d_weights=self.d_up, pre=self.pre,
                                 activation="silu", gated=True)
        e.combine_weighted(self.d_received, self.splits, self.keys, self.pos, K, None, self.d_x,
                           residual=dy)
        d_logits = [torch.empty_like(t) for t in self.logits]
        e.route_backward(self.logits, self.keys, self.d_weights, d_logits, self.k, score=self.score)
        self.d_gate = sum(d.T @ t.float() for d, t in zip(d_logits, self.x))
        for d, t in zip(d_logits, self.d_x):
            t += (d @ self.gate).to(t.dtype)
        return self.d_x


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--ranks", type=int, default=8)
    p.add_argument("--tokens", type=int, default=1024, help="of each rank")
    p.add_argument("--hidden", type=int, default=7168)
    p.add_argument("--inner", type=int, default=2048)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--topk", type=int, default=2)
    p.add_argument("--steps", type=int, default=10)
    a = p.parse_args()
    layer = MoeLayer(a.ranks, a.tokens, a.hidden, a.inner, a.experts, a.topk,
                     capacity=2 * a.tokens * a.topk)
    x = [torch.randn(a.tokens, a.hidden, device="cuda").bfloat16() for _ in range(a.ranks)]
    dy = [torch.randn_like(t) for t in x]
    for what, step in (("forward", lambda: layer.forward(x)),
                       ("forward and backward", lambda: (layer.forward(x), layer.backward(dy)))):
        for _ in range(3):
            step()
        assert layer.engine.status() == a2av.OK
        start = time.perf_counter()
        for _ in range(a.steps):
            step()
        assert layer.engine.status() == a2av.OK  # waits for the stream
        seconds = (time.perf_counter() - start) / a.steps
        print(f"{what}: {seconds * 1e3:.3f} ms, {a.ranks * a.tokens / seconds:.0f} tokens/s")


if __name__ == "__main__":
    main()
