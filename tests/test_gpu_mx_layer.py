"""The norm and the packed operators as they are used together: the block of
examples/moe_serving.py against 64 bits, and the norm in front of the layer of
examples/moe_layer.py, forward and backward, against automatic differentiation."""
import os
import sys

import pytest
import torch

from tests import _mx as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()


def _values(rows, D, fmt):
    """What packed rows stand for, in 64 bits."""
    v = mx.unpack(rows.reshape(-1, rows.shape[-1]).cpu().numpy(), D, fmt)[0]
    return torch.from_numpy(v).cuda().view(*rows.shape[:-1], D)


def _off(got, ref):
    return ((got.double() - ref).norm() / ref.norm().clamp_min(1e-30)).item()


def _answer(block, y):
    """What the experts add for each rank's rows y (64 bits: what the packed rows stand for), the
    block's own roundings of the inner activations made as well."""
    out = []
    up = [_values(t, block.H, block.format) for t in block.up]
    down = [_values(t, block.N, block.format) for t in block.down]
    for r in range(block.W):
        w = torch.softmax(block.logits[r].double().gather(1, block.keys[r].long()), 1)
        total = torch.zeros_like(y[r])
        for j in range(block.k):
            for e in range(block.E):
                t = (block.keys[r][:, j] == e).nonzero().reshape(-1)
                p, q = divmod(e, block.K)
                z = y[r][t] @ up[p][q].T
                a = (torch.nn.functional.silu(z[:, :block.N]) * z[:, block.N:]).to(block.dtype)
                packed = torch.from_numpy(mx.pack(a.double().cpu().numpy(), block.format)).cuda()
                total[t] += w[t, j][:, None] * (_values(packed, block.N, block.format) @ down[p][q].T)
        out.append(total)
    return out


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("shape", [(1, 5, 64, 32, 4, 2), (4, 33, 128, 72, 8, 2), (2, 40, 160, 64, 6, 3),
                                   (8, 16, 256, 128, 16, 4), (2, 1, 100, 64, 2, 1)])
def test_serving_block(shape, fmt):
    from moe_serving import PackedMoeBlock
    torch.manual_seed(0)
    block = PackedMoeBlock(*shape, format=fmt)
    x = [torch.randn(block.T, block.H, device="cuda").bfloat16() for _ in range(block.W)]
    h = [torch.randn_like(t) for t in x]
    sums = [(a.float() + b.float()).bfloat16() for a, b in zip(x, h)]
    kept = [t.clone() for t in h]
    block.forward(x, h)
    assert block.engine.status() == a2av.OK
    y = [_values(t, block.H, fmt) for t in block.packed]
    want = _answer(block, y)
    for r in range(block.W):
        exact = sums[r].double() / (sums[r].double().square().mean(1, keepdim=True) + block.eps).sqrt()
        # rounded once, to 8 bits; and to codes, each within half its step of the scaled value
        assert _off(block.y[r], exact) <= 2.0 ** -8
        rel, low = mx.HALF[fmt]
        scale = torch.from_numpy(mx.unpack(block.packed[r].cpu().numpy(), block.H, fmt)[1]).cuda()
        assert ((y[r] - exact).abs() <= torch.maximum(rel * exact.abs(), low * scale) * (1 + 1e-4)).all()
        ids = torch.sort(block.logits[r], dim=1, descending=True, stable=True).indices[:, :block.k]
        assert torch.equal(ids.int(), block.keys[r])
        # the answers and their sum with h are rounded to 8 bits; an inner value whose 32-bit sum
        # falls on the other side of a rounding's border (2^-24 of its terms against steps of 2^-8)
        # changes a code by a step: a hundredth of the answer's norm holds a dozen of those
        ref = sums[r].double() + want[r]
        assert (h[r].double() - ref).norm() <= 2.0 ** -8 * (ref.norm() + want[r].norm()) + 0.01 * want[r].norm()
    # the same as a graph, to the bit, whatever the buffers held
    again, first = [t.clone() for t in kept], [t.clone() for t in h]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x, again)
    for a, b in zip(again, kept):
        a.copy_(b)
    for t in block.packed + block.received + block.inner_packed:
        t.random_(0, 255)
    graph.replay()
    assert block.engine.status() == a2av.OK
    assert all(torch.equal(a, b) for a, b in zip(again, first))
    block.engine.close()


# one rounding more on the way there (y) and on the way back than the layer alone has
@pytest.mark.parametrize("dtype,limit", [(torch.bfloat16, 8 * 2.0 ** -8), (torch.float16, 8 * 2.0 ** -11)])
@pytest.mark.parametrize("shape", [(4, 33, 128, 72, 8, 2), (2, 100, 136, 64, 6, 3)])
def test_norm_before_the_layer(shape, dtype, limit):
    """h = x + residual, z = layer(norm(h)): the gradients of x, of the norm's weight and of what
    the layer holds, with h reaching the loss beside z."""
    from moe_layer import MoeLayer
    from tests.test_gpu_moe_layer import _reference
    torch.manual_seed(2)
    layer = MoeLayer(*shape, dtype=dtype)
    W, T, H, eps = layer.W, layer.T, layer.H, 1e-5
    new = lambda: [torch.randn(T, H, device="cuda").to(dtype) for _ in range(W)]
    x, residual, d_z, d_h = new(), new(), new(), new()
    weight = 1 + 0.2 * torch.randn(H, device="cuda")
    h, y, d_x, d_weight = new(), new(), new(), torch.empty(H, device="cuda")
    eng = layer.engine
    eng.norm(x, weight, y, residual=residual, sums=h, eps=eps)
    z = [t.clone() for t in layer.forward(y)]
    d_y = layer.backward(d_z)
    eng.norm_backward(h, weight, d_y, d_x, d_weight=d_weight, d_sums=d_h, eps=eps)
    assert eng.status() == a2av.OK
    # the layer's own gradient in 64 bits at y, and autograd of the norm before it
    zs, d_ys, *_ = _reference(layer, y, d_z)
    ws = weight.double().requires_grad_()
    hs = [t.double().requires_grad_() for t in h]
    loss = 0
    for r in range(W):
        assert torch.equal(h[r], (x[r].float() + residual[r].float()).to(dtype))
        n = hs[r] / (hs[r].square().mean(1, keepdim=True) + eps).sqrt() * ws
        assert _off(y[r], n.detach()) <= 2.0 ** (-8 if dtype == torch.bfloat16 else -11)
        assert _off(z[r], zs[r]) < limit
        loss = loss + (n * d_ys[r]).sum() + (hs[r] * d_h[r].double()).sum()
    loss.backward()
    for r in range(W):
        assert _off(d_x[r], hs[r].grad) < limit
    assert _off(d_weight, ws.grad) < limit
    layer.engine.close()
