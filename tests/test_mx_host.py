"""The norm's and the packed rows' calls without a GPU: sizes, what the library
refuses before any CUDA call, and the reference that the GPU tests use."""
import numpy as np
import pytest

import variable_size_all_gb300 as a2av
from tests import _mx as mx


@pytest.fixture(scope="module", autouse=True)
def _built():
    a2av.build()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("D", [1, 31, 32, 33, 64, 100, 1001, 2048, 7168, 1 << 24])
def test_row_bytes(D, fmt):
    assert a2av.mx_row_bytes(D, fmt) == mx.layout(D, fmt)[2]
    assert a2av.mx_row_bytes(D, fmt) % 32 == 0


def test_row_bytes_refusals():
    for D, f in ((0, a2av.MXFP8), (-1, a2av.MXFP4), ((1 << 24) + 1, a2av.MXFP8), (32, a2av.PLAIN), (32, 3)):
        assert a2av.a2av_mx_row_bytes(D, f) == -1
    for D, f in ((0, "mxfp8"), (32, None), (32, "fp8")):
        with pytest.raises(ValueError):
            a2av.mx_row_bytes(D, f)


def test_workspace_bytes():
    assert a2av.a2av_norm_workspace_bytes(100, 7) == 7 * 400
    assert a2av.a2av_norm_workspace_bytes(100, 1 << 30) == a2av.a2av_norm_workspace_bytes(100, 1 << 20)
    assert a2av.a2av_norm_workspace_bytes(100, 0) == 0
    for H, rows in ((0, 1), (a2av.MAX_NORM_FEATURES + 1, 1), (8, -1), (8, 1 << 31)):
        assert a2av.a2av_norm_workspace_bytes(H, rows) == -1


def test_calls_without_a_handle_are_refused():
    assert a2av.a2av_norm(None, 8, a2av.F32, a2av.PLAIN, 1e-6, [0], [1], 0, None, None, [0]) == a2av.ERR_INVALID_ARG
    assert a2av.a2av_norm_backward(None, 8, a2av.F32, 1e-6, [0], [1], 0, [0], None, [0], 0, 0, 0) == a2av.ERR_INVALID_ARG
    assert a2av.a2av_quantise(None, 8, a2av.F32, a2av.MXFP8, [0], [1], [0]) == a2av.ERR_INVALID_ARG
    assert a2av.a2av_dequantise(None, 8, a2av.F32, a2av.MXFP8, [0], [1], [0]) == a2av.ERR_INVALID_ARG
    shape = a2av.A2avExpert(1, 32, 8, a2av.BF16, 0, 0)
    assert a2av.a2av_expert_matmul_mx(None, shape, a2av.MXFP8, [0], [1], 0, [0], None, None,
                                      [0]) == a2av.ERR_INVALID_ARG


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_reference_codes(fmt):
    """Every code comes back, midpoints go to the even one, and a block's largest value fits."""
    t = mx.TABLE[fmt]
    assert np.array_equal(mx.codes_of(t, fmt), np.arange(len(t)))
    mid = (t[1:] + t[:-1]) / 2
    even = np.arange(len(mid)) + np.arange(len(mid)) % 2
    assert np.array_equal(mx.codes_of(mid, fmt), even)
    assert np.array_equal(mx.codes_of(-mid, fmt), even + (8 if fmt == "mxfp4" else 128))
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 70)) * 2.0 ** rng.integers(-30, 30, (50, 1))
    rows = mx.pack(x, fmt)
    v, scale = mx.unpack(rows, 70, fmt)
    rel, low = mx.HALF[fmt]
    assert (np.abs(v - x) <= np.maximum(rel * np.abs(x), low * scale)).all()
    top = np.abs(mx.blocks_of(x)).max(-1)
    s = mx.scales_of(mx.blocks_of(x), fmt)
    assert (top <= mx.MOST[fmt] * 2.0 ** (s - 127.0)).all()
    assert (top > mx.MOST[fmt] * 2.0 ** (s - 128.0)).all()


def test_reference_gradient_against_differences():
    rng = np.random.default_rng(1)
    s, w, dy = rng.standard_normal((3, 17)), rng.standard_normal(17), rng.standard_normal((3, 17))
    d, dw, _ = mx.norm_backward(s, w, dy, 1e-3)
    h = 1e-6
    for i in np.ndindex(s.shape):
        e = np.zeros_like(s)
        e[i] = h
        diff = ((mx.norm(s + e, w, 1e-3) - mx.norm(s - e, w, 1e-3)) * dy).sum() / (2 * h)
        assert abs(diff - d[i]) < 1e-7
    for j in range(17):
        e = np.zeros(17)
        e[j] = h
        diff = ((mx.norm(s, w + e, 1e-3) - mx.norm(s, w - e, 1e-3)) * dy).sum() / (2 * h)
        assert abs(diff - dw.sum(0)[j]) < 1e-7
