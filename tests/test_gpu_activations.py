"""The experts' activations and their slopes, one value at a time: at infinities
and NaN, and far down their tails, where the results are small."""
import math

import numpy as np
import pytest
import torch

from tests import _moe as moe

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()


def _forward(name, z, gated=False):
    """act(z) by the epilogue: the bias is z and the rows are zeros (one row of one expert)."""
    N, D = z.numel(), 8 if z.numel() % 8 == 0 else 5
    bias = torch.cat([z, torch.ones_like(z)]) if gated else z
    w = torch.zeros(1, bias.numel(), D, dtype=z.dtype, device="cuda")
    out = torch.empty(1, N, dtype=z.dtype, device="cuda")
    with a2av.A2av(1) as eng:
        eng.expert_matmul([torch.zeros(1, D, dtype=z.dtype, device="cuda")],
                          torch.ones(1, 1, dtype=torch.int64, device="cuda"), [w], [out],
                          activation=name, gated=gated, bias=[bias.view(1, -1)])
        assert eng.status() == a2av.OK
    return out[0].double().cpu().numpy()


def _slope(name, z, gated=False):
    """act'(z), and act(z) of the gate, as the gradient of the bias (dy = 1, the partners are 1)."""
    N, D = z.numel(), 8
    pre = torch.cat([z, torch.ones_like(z)]) if gated else z
    w = torch.zeros(1, pre.numel(), D, dtype=z.dtype, device="cuda")
    d_bias = torch.empty(1, pre.numel(), dtype=z.dtype, device="cuda")
    with a2av.A2av(1) as eng:
        eng.expert_matmul_backward([torch.zeros(1, D, dtype=z.dtype, device="cuda")],
                                   torch.ones(1, 1, dtype=torch.int64, device="cuda"), [w],
                                   [torch.ones(1, N, dtype=z.dtype, device="cuda")], d_bias=[d_bias],
                                   pre=[pre.view(1, -1)], activation=name, gated=gated)
        assert eng.status() == a2av.OK
    return d_bias[0].double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("size", [8, 7])
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu"])
def test_infinities_and_nan(name, size, gated, dtype):
    """An activation at an infinity is its limit, and so is its slope: a row whose
    pre-activation is out of the type's range still has a gradient.  NaN stays."""
    inf, nan, big = math.inf, math.nan, torch.finfo(dtype).max
    z = torch.tensor(([inf, -inf, nan, big, -big, 0.0, 300.0, -300.0])[:size], dtype=dtype, device="cuda")
    x = z.double().cpu().numpy()
    up = x if name == "none" else np.where(x < 0, 0.0, x)
    slope = np.ones(size) if name == "none" else (x > 0) * 1.0
    if name in ("gelu", "silu"):
        slope = np.where(x == 0, 0.5, slope)
    assert np.array_equal(_forward(name, z, gated), up, equal_nan=True)
    got = _slope(name, z, gated)
    if name in ("gelu", "silu"):
        slope = np.where(np.isnan(x), nan, slope)
    known = ~np.isnan(x) | np.isin(name, ["gelu", "silu"])  # (a step's slope at NaN is anything)
    assert np.array_equal(got[:size][known], slope[known], equal_nan=True)
    if gated:
        assert np.array_equal(got[size:], up, equal_nan=True)


def _exact(name, x):
    """(act, slope, the magnitude of the slope's terms) in 64 bits, without cancellation."""
    phi = np.array([0.5 * math.erfc(-v / math.sqrt(2)) for v in x])
    dens = np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if name == "gelu":
        return x * phi, phi + x * dens, phi + np.abs(x) * dens
    s, c = 1 / (1 + np.exp(-x)), 1 / (1 + np.exp(x))
    return x * s, s * (1 + x * c), s * (1 + np.abs(x) * c)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_small_results_are_as_exact_as_large_ones(name, dtype):
    """Relative error over the whole range: the rounding to the type, and 2^-16 for
    the arithmetic before it.  (The exponential's argument, at most z^2 / 2 log2(e)
    = 75 for the z below and rounded three times, is the most of that: 75 * 3 *
    2^-24 * ln 2 = 2^-17.)"""
    z = torch.cat([torch.linspace(-10.2, 10.2, 4096), torch.linspace(-1, 1, 512),
                   torch.logspace(-6, 0, 256, 10.0), -torch.logspace(-6, 0, 256, 10.0)])
    z = z.to(moe.DTYPES[dtype]).cuda()
    act, slope, size = _exact(name, z.double().cpu().numpy())
    moe.close(_forward(name, z), act, 2.0 ** -16 * np.abs(act), dtype, name)
    moe.close(_slope(name, z), slope, 2.0 ** -16 * size, dtype, f"{name}'s slope")
