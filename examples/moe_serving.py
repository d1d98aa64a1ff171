"""The MoE block of a decoder for serving, on W ranks, its rows and experts' weights packed.

    python examples/moe_serving.py [--format mxfp4] [--tokens 16] [--hidden 7168] ...

Each rank has its tokens' residual stream h [T, H] and what the block before adds
to it, x [T, H]:

    h = h + x;  y = norm(h)
    h' = h + sum_j weight_j * (silu(y Wg^T) * (y Wu^T)) Wd^T        (expert j's weights)

The norm writes y as packed rows (8 or 4 bits and a scale for each 32 values), which
go through the exchange as they are, and in 16 bits for the router.  The experts'
products take packed rows and weights; between the two the inner activations are
packed again.  No call waits for the device, so a step can be captured into a graph.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import variable_size_all_gb300 as a2av  # noqa: E402


class PackedMoeBlock:
    """Packed weights, buffers and the forward pass.  ``capacity``: rows a rank can
    receive (a dispatch of more is refused on the device)."""

    def __init__(self, W, tokens, hidden, inner, experts, topk, format="mxfp8", dtype=torch.bfloat16,
                 capacity=None, eps=1e-6):
        self.W, self.T, self.H, self.N, self.k, self.eps = W, tokens, hidden, inner, topk, eps
        self.E, self.K, self.format, self.dtype = experts, experts // W, format, dtype
        self.capacity = C = capacity or W * tokens * topk
        self.engine = a2av.A2av(W, out_capacity_rows=C)
        self.row, self.inner_row = a2av.mx_row_bytes(hidden, format), a2av.mx_row_bytes(inner, format)
        new = lambda *shape, dtype=dtype: [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(W)]
        K, T, H, N, k = self.K, tokens, hidden, inner, topk
        self.norm_weight = torch.ones(H, device="cuda")
        self.gate = torch.randn(experts, H, device="cuda") * H ** -0.5
        self.up, self.down = self.pack(2 * N, H), self.pack(H, N)
        self.y, self.packed = new(T, H), new(T, self.row, dtype=torch.uint8)
        self.keys, self.weights = new(T, k, dtype=torch.int32), new(T, k, dtype=torch.float32)
        self.counts = torch.empty(W, experts, dtype=torch.int64, device="cuda")
        self.splits = torch.empty(W, W, dtype=torch.int64, device="cuda")
        self.offsets = torch.empty(W, 2, W, dtype=torch.int64, device="cuda")
        self.pos = new(T * k, dtype=torch.int64)
        self.source = [torch.arange(T, dtype=torch.int32, device="cuda").repeat_interleave(k)
                       for _ in range(W)]
        self.received = new(C, self.row, dtype=torch.uint8)
        self.inner, self.answer = new(C, N), new(C, H)
        self.inner_packed = new(C, self.inner_row, dtype=torch.uint8)

    def pack(self, features, width):
        """Random weights [K, features, width] of each rank, packed expert by expert."""
        packed = [torch.empty(self.K, features, a2av.mx_row_bytes(width, self.format), dtype=torch.uint8,
                              device="cuda") for _ in range(self.W)]
        for e in range(self.K):
            w = [(torch.randn(features, width, device="cuda") * width ** -0.5).to(self.dtype)
                 for _ in range(self.W)]
            self.engine.quantise(w, [p[e] for p in packed], self.format)
        return packed

    def forward(self, x, h):
        """Adds x and the experts' answers to h, in place."""
        e, K = self.engine, self.K
        e.norm(x, self.norm_weight, self.packed, residual=h, sums=h, eps=self.eps, format=self.format,
               plain=self.y)
        # the gate's product is a small dense one
        self.logits = [t.float() @ self.gate.T for t in self.y]
        e.route(self.logits, self.keys, self.weights, self.k, counts=self.counts)
        e.dispatch(self.packed, self.source, [t.view(-1) for t in self.keys], K, self.received,
                   self.offsets, self.pos, self.row, in_splits=self.splits)
        e.expert_matmul_mx(self.received, self.counts, self.up, self.inner, self.H, self.format,
                           activation="silu", gated=True)
        e.quantise(self.inner, self.inner_packed, self.format, in_splits=self.splits)
        e.expert_matmul_mx(self.inner_packed, self.counts, self.down, self.answer, self.N, self.format)
        e.combine_weighted(self.answer, self.splits, self.keys, self.pos, K, self.weights, h, residual=h)
        return h


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--format", choices=("mxfp8", "mxfp4"), default="mxfp4")
    p.add_argument("--ranks", type=int, default=8)
    p.add_argument("--tokens", type=int, default=16, help="of each rank")
    p.add_argument("--hidden", type=int, default=7168)
    p.add_argument("--inner", type=int, default=2048)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--topk", type=int, default=2)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    block = PackedMoeBlock(a.ranks, a.tokens, a.hidden, a.inner, a.experts, a.topk, a.format)
    x = [torch.randn(a.tokens, a.hidden, device="cuda").bfloat16() for _ in range(a.ranks)]
    h = [torch.randn_like(t) for t in x]
    for _ in range(3):
        block.forward(x, h)
    assert block.engine.status() == a2av.OK
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x, h)
    for what, step in (("call by call", lambda: block.forward(x, h)), ("as a graph", graph.replay)):
        step()
        assert block.engine.status() == a2av.OK
        start = time.perf_counter()
        for _ in range(a.steps):
            step()
        assert block.engine.status() == a2av.OK  # waits for the stream
        seconds = (time.perf_counter() - start) / a.steps
        print(f"{what}: {seconds * 1e3:.3f} ms, {a.ranks * a.tokens / seconds:.0f} tokens/s")


if __name__ == "__main__":
    main()
