"""The gradient of sigmoid scores that are almost 1, or almost 0."""
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


@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_saturated_scores(renorm):
    """s (1 - s) of a sigmoid near 1: 1 - s is 1 / (1 + exp(x)), not what is left of
    a difference.  Relative error 2^-19: the exponential's 2 ulp, the rounding of
    s, of the products and (renormalised) of two quotients and a difference of
    numbers that are not near each other."""
    x = torch.tensor([[v, -v / 2, 1.0, -2.0] for v in np.linspace(-20, 25, 181)], dtype=torch.float32,
                     device="cuda")
    keys = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda").repeat(181, 1)
    g = torch.tensor([[1.0, -2.0, 0.25]], device="cuda").repeat(181, 1)
    d = torch.empty_like(x)
    with a2av.A2av(1) as eng:
        eng.route_backward([x], [keys], [g], [d], 3, score="sigmoid", renormalise=renorm)
        assert eng.status() == a2av.OK
    x64, s = moe.f64(x)[:, :3], 1 / (1 + np.exp(-moe.f64(x)[:, :3]))
    c, g64 = 1 / (1 + np.exp(x64)), moe.f64(g)
    size = np.abs(g64)
    if renorm:
        t = s.sum(1, keepdims=True)
        g64, size = (g64 - (g64 * s).sum(1, keepdims=True) / t) / t, (size + (size * s).sum(1, keepdims=True) / t) / t
    assert (np.abs(moe.f64(d)[:, :3] - g64 * s * c) <= 2.0 ** -19 * size * s * c + 2.0 ** -126).all()
    assert not d[:, 3].any()
