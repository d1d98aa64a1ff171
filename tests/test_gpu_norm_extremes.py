"""The norm and its gradients at the ends of their ranges: infinite weights, rows
whose squares leave 32 bits on either side, the largest eps."""
import numpy as np
import pytest
import torch

from tests import _moe as moe
from tests import _mx as mx

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()


def _place(values, dtype):
    return torch.from_numpy(np.ascontiguousarray(values)).to(moe.DTYPES[dtype]).cuda()


def _norm(x, w, eps, fmt=None, plain=None):
    width = x.shape[1] if fmt is None else a2av.mx_row_bytes(x.shape[1], fmt)
    out = torch.empty(x.shape[0], width, dtype=x.dtype if fmt is None else torch.uint8, device="cuda")
    with a2av.A2av(1) as eng:
        eng.norm([x], w, [out], eps=eps, format=fmt, plain=None if plain is None else [plain])
        assert eng.status() == a2av.OK
    return out


def _norm_backward(s, w, dy, eps, ds=None):
    dx, dw = torch.empty_like(s), torch.empty(s.shape[1], device="cuda")
    with a2av.A2av(1) as eng:
        eng.norm_backward([s], w, [dy], [dx], d_weight=dw, d_sums=None if ds is None else [ds], eps=eps)
        assert eng.status() == a2av.OK
    return dx, dw


# a warp a row, a block a row, rows of no vectors, many rows (fetched ahead)
SHAPES = [(5, 256), (3, 2048), (3, 1001), (1, 33), (5000, 512), (900, 7168)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_weights_without_end(shape, dtype):
    """An infinite or NaN weight: the product's infinity (NaN for 0), in its own column;
    its block of a packed row is NaN, the others are what they were."""
    T, H = shape
    rng = np.random.default_rng(H)
    values = rng.standard_normal((T, H))
    values[0, 3] = 0.0
    x, w = _place(values, dtype), torch.from_numpy(1 + 0.3 * rng.standard_normal(H)).float().cuda()
    odd = torch.tensor([0, 3, 5, H - 1], device="cuda")
    bad = w.clone()
    bad[odd] = torch.tensor([np.inf, np.inf, np.nan, -np.inf], device="cuda")
    rest = torch.ones(H, dtype=torch.bool, device="cuda")
    rest[odd] = False
    clean, out = _norm(x, w, 1e-5), _norm(x, bad, 1e-5)
    assert torch.equal(out[:, rest], clean[:, rest])
    ref = mx.norm(moe.f64(x), moe.f64(bad), 1e-5)[:, odd.cpu().numpy()]
    assert np.array_equal(moe.f64(out[:, odd]), ref, equal_nan=True)
    for fmt in ("mxfp8", "mxfp4"):
        plain = torch.empty_like(x)
        a, b = _norm(x, w, 1e-5, fmt), _norm(x, bad, 1e-5, fmt, plain)
        assert torch.equal(plain.nan_to_num(9), out.nan_to_num(9))
        v, u = mx.unpack(a.cpu().numpy(), H, fmt)[0], mx.unpack(b.cpu().numpy(), H, fmt)[0]
        lost = np.isin(np.arange(H) // 32, odd.cpu().numpy() // 32)
        assert np.isnan(u[:, lost]).all() and np.array_equal(u[:, ~lost], v[:, ~lost])


@pytest.mark.parametrize("more", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients_of_long_rows(shape, dtype, more):
    """Rows whose squares pass 2^128 count as of infinite length: nothing reaches them
    but d_sums, also where the products' sum passes it too; other rows are as alone."""
    T, H = shape
    rng = np.random.default_rng(H + 1)
    values, up = rng.standard_normal((T + 3, H)), rng.standard_normal((T + 3, H))
    values[1], up[1] = 3e38, 1e3
    values[2] = np.where(np.arange(H) % 2, -1e30, 1e30)
    values[T + 2, 1], values[T + 2, 2] = np.inf, 2.0
    s, dy, w = _place(values, dtype), _place(up, dtype), torch.ones(H, device="cuda")
    ds = _place(rng.standard_normal((T + 3, H)), dtype) if more else None
    dx, dw = _norm_backward(s, w, dy, 1e-5, ds)
    still = ds if more else torch.zeros_like(s)
    assert torch.equal(dx[1:3], still[1:3])
    finite = torch.ones(H, dtype=torch.bool, device="cuda")
    finite[1] = False
    assert torch.equal(dx[-1][finite], still[-1][finite]) and dx[-1, 1].isnan()
    kept = torch.ones(T + 3, dtype=torch.bool, device="cuda")
    kept[[1, 2, T + 2]] = False
    d, terms, size = mx.norm_backward(moe.f64(s[kept]), np.ones(H), moe.f64(dy[kept]), 1e-5)
    bound = 4 * mx.norm_error(H) * size
    if more:
        d = d + moe.f64(ds[kept])
        bound = bound + 2.0 ** -24 * np.abs(d)
    moe.close(dx[kept], d, bound, dtype, "d_x")
    at = finite.cpu().numpy()
    moe.close(moe.f64(dw)[at], terms.sum(0)[at],
              ((4 * mx.norm_error(H) + (T + 8) * 2.0 ** -24) * np.abs(terms).sum(0))[at], "f32", "d_weight")
    assert dw[1].isnan()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_short_rows_without_eps(shape, dtype):
    """eps = 0 and values of 2^-66, whose squares 32 bits hold exactly: 1 / rms^2 does not
    fit in them, the results do."""
    T, H = shape
    rng = np.random.default_rng(H + 2)
    s = _place(rng.choice([-1.0, 1.0], (T, H)) * 2.0 ** -66, dtype)
    dy, w = _place(rng.standard_normal((T, H)), dtype), torch.from_numpy(rng.uniform(0.5, 1.5, H)).float().cuda()
    y = mx.norm(moe.f64(s), moe.f64(w), 0.0)
    moe.close(_norm(s, w, 0.0), y, mx.norm_error(H) * np.abs(y), dtype, "y")
    dx, dw = _norm_backward(s, w, dy, 0.0)
    d, terms, size = mx.norm_backward(moe.f64(s), moe.f64(w), moe.f64(dy), 0.0)
    moe.close(dx, d, 4 * mx.norm_error(H) * size, dtype, "d_x")
    moe.close(dw, terms.sum(0), (4 * mx.norm_error(H) + (T + 8) * 2.0 ** -24) * np.abs(terms).sum(0), "f32",
              "d_weight")


def test_no_length_at_all():
    """eps = 0 and rows whose squares are 0 in 32 bits."""
    s = torch.zeros(3, 64, device="cuda")
    s[1], s[2, 0] = 1e-30, -1e-30
    assert _norm(s, torch.ones(64, device="cuda"), 0.0).isnan().all()


def test_largest_eps():
    eps = float(np.finfo(np.float32).max)
    x, w = torch.randn(7, 96, device="cuda"), torch.ones(96, device="cuda")
    y = mx.norm(moe.f64(x), moe.f64(w), eps)
    moe.close(_norm(x, w, eps), y, mx.norm_error(96) * np.abs(y), "f32", "y")
    dx, _ = _norm_backward(x, w, x, eps)
    d, _, size = mx.norm_backward(moe.f64(x), moe.f64(w), moe.f64(x), eps)
    moe.close(dx, d, 4 * mx.norm_error(96) * size, "f32", "d_x")
