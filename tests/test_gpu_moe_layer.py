"""The MoE layer of examples/moe_layer.py, forward and backward, against torch's
automatic differentiation in 64 bits, with the routing that the layer chose."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()


def _reference(layer, x, dy):
    """y and the gradients, by autograd in 64 bits (the choice of experts is given)."""
    xs = [t.double().requires_grad_() for t in x]
    gate = layer.gate.double().requires_grad_()
    up = [t.double().requires_grad_() for t in layer.up]
    down = [t.double().requires_grad_() for t in layer.down]
    loss, ys = 0, []
    for r in range(layer.W):
        ids = layer.keys[r].long()
        score = (xs[r] @ gate.T).gather(1, ids)
        w = torch.softmax(score, 1) if layer.score == "softmax" else \
            torch.sigmoid(score) / torch.sigmoid(score).sum(1, keepdim=True)
        y = xs[r]
        for e in range(layer.E):
            t, j = (ids == e).nonzero(as_tuple=True)
            p, q = divmod(e, layer.K)
            z = xs[r][t] @ up[p][q].T
            h = torch.nn.functional.silu(z[:, :layer.N]) * z[:, layer.N:]
            y = y.index_add(0, t, w[t, j][:, None] * (h @ down[p][q].T))
        ys.append(y.detach())
        loss = loss + (y * dy[r].double()).sum()
    loss.backward()
    return ys, [t.grad for t in xs], gate.grad, [t.grad for t in up], [t.grad for t in down]


def _off(got, ref):
    return ((got.double() - ref).norm() / ref.norm().clamp_min(1e-30)).item()


# a chain of roundings to 8 or 11 bits (received rows, pre, inner, answer and their gradients):
# each adds at most 2^-8 or 2^-11 of the values' norm, six of them in a row
@pytest.mark.parametrize("dtype,limit", [(torch.bfloat16, 6 * 2.0 ** -8), (torch.float16, 6 * 2.0 ** -11)])
@pytest.mark.parametrize("shape", [(1, 5, 64, 32, 4, 2), (4, 33, 128, 72, 8, 2), (2, 100, 136, 64, 6, 3),
                                   (8, 16, 256, 128, 16, 4), (2, 1, 64, 64, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_layer(shape, dtype, limit, score):
    from moe_layer import MoeLayer
    torch.manual_seed(0)
    layer = MoeLayer(*shape, dtype=dtype, score=score)
    x = [torch.randn(layer.T, layer.H, device="cuda").to(dtype) for _ in range(layer.W)]
    dy = [torch.randn_like(t) for t in x]
    y = layer.forward(x)
    d_x = layer.backward(dy)
    assert layer.engine.status() == a2av.OK
    ys, dxs, d_gate, d_up, d_down = _reference(layer, x, dy)
    for got, ref in list(zip(y, ys)) + list(zip(d_x, dxs)):
        assert _off(got, ref) < limit
    for got, ref in ((torch.stack(layer.d_up), torch.stack(d_up)),
                     (torch.stack(layer.d_down), torch.stack(d_down))):
        assert _off(got, ref) < limit
    if layer.k > 1:  # (a single renormalised weight is 1: no gradient)
        assert _off(layer.d_gate, d_gate) < 4 * limit
    layer.engine.close()


def test_capacity_is_kept():
    """More rows than the peers' buffers hold: refused on the device, nothing is run past the end."""
    from moe_layer import MoeLayer
    torch.manual_seed(1)
    layer = MoeLayer(2, 64, 64, 32, 4, 2, capacity=64)
    x = [torch.randn(64, 64, device="cuda").bfloat16() for _ in range(2)]
    layer.forward(x)
    assert layer.engine.status() == a2av.ERR_BAD_SPLITS
    layer.engine.close()
