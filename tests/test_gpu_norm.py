"""The norm and its gradients on the GPU against the definition in 64 bits, with
error bounds from the arithmetic, and what they refuse."""
import numpy as np
import pytest
import torch

from tests import _moe as moe
from tests import _mx as mx

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()


def _place(values, dt, offset=0):
    buf = torch.empty(values.size + offset, dtype=dt, device="cuda")
    view = buf[offset:].view(values.shape)
    view.copy_(torch.from_numpy(np.ascontiguousarray(values)))
    return view


def _rows(tokens, H, dtype, seed, offset=0, std=1.0):
    rng = np.random.default_rng(seed)
    return [_place(rng.standard_normal((t, H)) * std * 2.0 ** rng.integers(-3, 4, (t, 1)), moe.DTYPES[dtype], offset)
            for t in tokens]


def _weight(H, seed=9):
    return _place(1 + 0.3 * np.random.default_rng(seed).standard_normal(H), torch.float32)


def _check_rows(got, y, w, fmt, dtype, what):
    """Rows of y, 64 bits, against what the kernel wrote."""
    H = y.shape[1]
    error = mx.norm_error(H)
    if fmt is None:
        return moe.close(got, y, error * np.abs(y), dtype, what)
    rows = got.cpu().numpy()
    V, B, _ = mx.layout(H, fmt)
    assert (rows[:, V + B:] == 0).all(), "bytes behind the scales"
    whole = mx.unpack(rows, 32 * B, fmt)[0]
    assert (whole[:, H:] == 0).all(), "values behind the row"
    v, scale = mx.unpack(rows, H, fmt)
    top = np.abs(mx.blocks_of(y)).max(-1)
    s = 2.0 ** (rows[:, V:V + B].astype(np.float64) - 127)
    assert (top * (1 - error) <= mx.MOST[fmt] * s).all(), "scales too small"
    assert ((top * (1 + error) >= mx.MOST[fmt] * s / 2) | (s == 2.0 ** -127)).all(), "scales too large"
    rel, low = mx.HALF[fmt]
    limit = np.maximum(rel * np.abs(y), low * scale) * (1 + error) + error * np.abs(y)
    assert (np.abs(v - y) <= limit * (1 + 1e-9)).all(), what


def _forward(x, w, dtype, res=None, sums=None, fmt=None, eps=EPS, stream=None):
    W, H = len(x), x[0].shape[1]
    if fmt is None:
        out = [torch.full_like(t, 7) for t in x]
    else:
        out = [torch.full((t.shape[0], a2av.mx_row_bytes(H, fmt)), 7, dtype=torch.uint8, device="cuda") for t in x]
    with a2av.A2av(W) as eng:
        eng.norm(x, w, out, residual=res, sums=sums, eps=eps, format=fmt, stream=stream)
        assert eng.status(stream) == a2av.OK
    return out


# (tokens of each rank, features): a warp a row, a block a row, rows of no vectors,
# fewer and more rows than a GPU holds at once, ranks without any
SHAPES = [([1], 1), ([3, 0, 5], 33), ([4], 32), ([2, 9], 64), ([17], 100), ([700, 1], 200), ([40], 512),
          ([5], 513), ([7], 1000), ([30, 31], 1001), ([1], 7168), ([4] * 8, 7168), ([500, 400], 2048),
          ([9], 4104), ([3], 16384), ([2], 16383), ([1200], 1504), ([0, 0], 64), ([400], 8192)]


@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm(shape, dtype, residual, fmt):
    tokens, H = shape
    x, w = _rows(tokens, H, dtype, 1), _weight(H)
    res = _rows(tokens, H, dtype, 2) if residual else None
    sums = [torch.full_like(t, 7) for t in x]
    out = _forward(x, w, dtype, res, sums, fmt)
    for r in range(len(tokens)):
        s = (x[r].float() + res[r].float()).to(x[r].dtype) if residual else x[r]
        assert torch.equal(sums[r], s)
        _check_rows(out[r], mx.norm(moe.f64(s), moe.f64(w), EPS), moe.f64(w), fmt, dtype, f"rank {r}")


@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("offset", [1, 3])
def test_unaligned_buffers(offset, fmt):
    for H in (96, 2048):
        x, res, w = _rows([6, 2], H, "bf16", 3, offset), _rows([6, 2], H, "bf16", 4, offset), _weight(H)
        sums = [_place(np.zeros((t, H)), torch.bfloat16, offset) for t in (6, 2)]
        out = _forward(x, w, "bf16", res, sums, fmt)
        for r in range(2):
            s = (x[r].float() + res[r].float()).bfloat16()
            assert torch.equal(sums[r], s)
            _check_rows(out[r], mx.norm(moe.f64(s), moe.f64(w), EPS), moe.f64(w), fmt, "bf16", f"rank {r}")


def test_sums_in_place():
    x, res, w = _rows([33], 640, "bf16", 5), _rows([33], 640, "bf16", 6), _weight(640)
    want = [torch.empty_like(t) for t in x]
    out = _forward(x, w, "bf16", res, want)
    for into in (x, res):
        a, b = [t.clone() for t in x], [t.clone() for t in res]
        kept = a if into is x else b
        again = _forward(a, w, "bf16", b, kept)
        assert torch.equal(kept[0], want[0]) and torch.equal(again[0], out[0])


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_packed_output_is_the_plain_ones(fmt):
    """In 32 bits the packed result is a2av_quantise's of the plain one, to the bit."""
    for H in (7168, 515):
        x, w = _rows([65], H, "f32", 7), _weight(H)
        plain, packed = _forward(x, w, "f32"), _forward(x, w, "f32", fmt=fmt)
        again = [torch.empty_like(packed[0])]
        with a2av.A2av(1) as eng:
            eng.quantise(plain, again, fmt)
            assert eng.status() == a2av.OK
        assert torch.equal(again[0], packed[0])


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_both_outputs(fmt):
    """With a packed result, the plain one as well: each what a call by itself gives."""
    for dtype, tokens, H, offset in (("bf16", [9, 0, 2], 1024, 0), ("f32", [3], 100, 0), ("f16", [700], 1504, 1),
                                     ("bf16", [900], 7168, 0)):
        x, res, w = _rows(tokens, H, dtype, 40, offset), _rows(tokens, H, dtype, 41, offset), _weight(H)
        want, packed = _forward(x, w, dtype, res), _forward(x, w, dtype, res, fmt=fmt)
        out, plain = [torch.zeros_like(t) for t in packed], [torch.zeros_like(t) for t in x]
        with a2av.A2av(len(x)) as eng:
            eng.norm(x, w, out, residual=res, eps=EPS, format=fmt, plain=plain)
            assert eng.status() == a2av.OK
            with pytest.raises(ValueError):
                eng.norm(x, w, plain, residual=res, plain=plain)
        assert all(torch.equal(a, b) for a, b in zip(out + plain, packed + want))


def test_special_rows():
    """Rows of zeros, of NaN and infinities, and rows whose squares pass 32 bits, by themselves."""
    H = 256
    x, w = _rows([6], H, "f32", 8), _weight(H)
    x[0][1] = 0
    x[0][2, 5] = float("nan")
    x[0][3, 7] = float("inf")
    x[0][4] = 3e38
    out = _forward(x, w, "f32")[0]
    assert (out[1] == 0).all() and out[2].isnan().all() and out[3, 7].isnan() and (out[4] == 0).all()
    y = mx.norm(moe.f64(x[0]), moe.f64(w), EPS)
    for t in (0, 5):
        moe.close(out[t], y[t], mx.norm_error(H) * np.abs(y[t]), "f32", f"row {t}")
    packed = _forward(x, w, "f32", fmt="mxfp8")[0].cpu().numpy()
    v = mx.unpack(packed, H, "mxfp8")[0]
    assert (v[1] == 0).all() and np.isnan(v[2]).all() and np.isnan(v[3, :32]).all() and (v[3, 32:] == 0).all()
    assert np.isfinite(v[[0, 4, 5]]).all()


def _backward(s, w, dy, ds, dx=None, dw=True, eps=EPS, stream=None, workspace=None):
    dx = [torch.full_like(t, 7) for t in s] if dx is None else dx
    d_weight = torch.full((s[0].shape[1],), 7.0, device="cuda") if dw else None
    with a2av.A2av(len(s)) as eng:
        eng.norm_backward(s, w, dy, dx, d_weight=d_weight, d_sums=ds, eps=eps, stream=stream,
                          workspace=workspace)
        assert eng.status(stream) == a2av.OK
    return dx, d_weight


def _check_backward(s, w, dy, ds, dx, dw, dtype, eps=EPS):
    H, terms, size = s[0].shape[1], np.zeros(s[0].shape[1]), np.zeros(s[0].shape[1])
    error = 4 * mx.norm_error(H)
    n = 0
    for r in range(len(s)):
        if s[r].shape[0] == 0:
            continue
        d, t, mag = mx.norm_backward(moe.f64(s[r]), moe.f64(w), moe.f64(dy[r]), eps)
        bound = error * mag
        if ds is not None:
            d = d + moe.f64(ds[r])
            bound = bound + 2.0 ** -24 * np.abs(d)
        moe.close(dx[r], d, bound, dtype, f"d_x of rank {r}")
        terms, size, n = terms + t.sum(0), size + np.abs(t).sum(0), n + s[r].shape[0]
    if dw is not None:
        moe.close(dw, terms, (error + (n + 8) * 2.0 ** -24) * size, "f32", "d_weight")


@pytest.mark.parametrize("more", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dtype, more):
    tokens, H = shape
    s, w = _rows(tokens, H, dtype, 11), _weight(H)
    dy, ds = _rows(tokens, H, dtype, 12), _rows(tokens, H, dtype, 13) if more else None
    dx, dw = _backward(s, w, dy, ds)
    _check_backward(s, w, dy, ds, dx, dw, dtype)
    only, none = _backward(s, w, dy, ds, dw=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip(only, dx))
    again, dw2 = _backward(s, w, dy, ds)
    assert torch.equal(dw, dw2), "the weight's gradient depends on the order of blocks"


def test_backward_unaligned_and_in_place():
    for H in (96, 2048):
        s, w = _rows([6, 2], H, "f16", 14, 1), _weight(H)
        dy, ds = _rows([6, 2], H, "f16", 15, 1), _rows([6, 2], H, "f16", 16, 1)
        dx, dw = _backward(s, w, dy, ds)
        _check_backward(s, w, dy, ds, dx, dw, "f16")
        for which in (0, 1):
            a, b = [t.clone() for t in dy], [t.clone() for t in ds]
            into, dw2 = _backward(s, w, a, b, dx=(a, b)[which])
            assert all(torch.equal(p, q) for p, q in zip(into, dx))
            torch.testing.assert_close(dw2, dw, rtol=1e-5, atol=1e-5)


def test_gradient_against_differences():
    """The kernel's gradient in 32 bits against central differences of the definition in 64."""
    H = 48
    s, w, dy = _rows([2], H, "f32", 17), _weight(H), _rows([2], H, "f32", 18)
    dx, dw = _backward(s, w, dy, None)
    x, g, d = moe.f64(s[0]), moe.f64(w), moe.f64(dy[0])
    h = 1e-6

    def f(x, g):
        return (mx.norm(x, g, EPS) * d).sum()

    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        diff = (f(x + e, g) - f(x - e, g)) / (2 * h)
        # differences: h^2 of the third derivative and 2^-53 / h of the sum; 32 bits as above
        assert abs(float(dx[0][i]) - diff) < 1e-4 * max(1.0, abs(diff))
    for j in range(H):
        e = np.zeros(H)
        e[j] = h
        diff = (f(x, g + e) - f(x, g - e)) / (2 * h)
        assert abs(float(dw[j]) - diff) < 1e-4 * max(1.0, abs(diff))


def test_graph_streams_and_bound_calls():
    """Captured and replayed on new values, on a side stream, and bound."""
    tokens, H = [5, 300], 1024
    x, res, w = _rows(tokens, H, "bf16", 20), _rows(tokens, H, "bf16", 21), _weight(H)
    dy = _rows(tokens, H, "bf16", 22)
    want = [torch.empty_like(t) for t in x]
    plain = _forward(x, w, "bf16", res, want)
    want_dx, want_dw = _backward(want, w, dy, res)
    out, sums, dx = ([torch.empty_like(t) for t in x] for _ in range(3))
    dw = torch.empty(H, device="cuda")
    side = torch.cuda.Stream()
    with a2av.A2av(2) as eng:
        side.wait_stream(torch.cuda.current_stream())
        eng.norm(x, w, out, residual=res, sums=sums, eps=EPS, stream=side)
        eng.norm_backward(sums, w, dy, dx, d_weight=dw, d_sums=res, eps=EPS, stream=side)
        assert eng.status(side) == a2av.OK
        assert all(torch.equal(a, b) for a, b in zip(out + dx + [dw], plain + want_dx + [want_dw]))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            eng.norm(x, w, out, residual=res, sums=sums, eps=EPS)
            eng.norm_backward(sums, w, dy, dx, d_weight=dw, d_sums=res, eps=EPS)
        for t in out + sums + dx + [dw]:
            t.zero_()
        # an eager call between two replays shares no workspace with the graph
        for _ in range(2):
            graph.replay()
            other = torch.empty(H, device="cuda")
            eng.norm_backward(want, w, dy, [torch.empty_like(t) for t in x], d_weight=other, d_sums=res, eps=EPS)
        torch.cuda.synchronize()
        assert torch.equal(other, want_dw)
        assert all(torch.equal(a, b) for a, b in zip(out + sums + dx + [dw], plain + want + want_dx + [want_dw]))
        call = eng.bind_norm(x, w, out, residual=res, sums=sums, eps=EPS)
        for t in x:
            t.mul_(2)
        call()
        assert eng.status() == a2av.OK
    s = (x[1].float() + res[1].float()).bfloat16()
    assert torch.equal(sums[1], s)
    _check_rows(out[1], mx.norm(moe.f64(s), moe.f64(w), EPS), moe.f64(w), None, "bf16", "bound")


def test_refusals():
    x, w = _rows([4], 64, "bf16", 30), _weight(64)
    out = [torch.empty_like(t) for t in x]
    packed = [torch.empty(4, a2av.mx_row_bytes(64, "mxfp8"), dtype=torch.uint8, device="cuda")]
    with a2av.A2av(1) as eng:
        for bad in (dict(weight=w.bfloat16()), dict(weight=w[:32]), dict(weight=w.cpu()),
                    dict(outputs=[out[0].float()]), dict(outputs=packed), dict(outputs=out, format="mxfp8"),
                    dict(residual=[x[0][:2]]), dict(sums=[x[0].float()]), dict(format="fp8"),
                    dict(x=[x[0].double()]), dict(x=x + x), dict(x=[x[0].t()]), dict(outputs=[None])):
            args = {"x": x, "weight": w, "outputs": out, **bad}
            with pytest.raises(ValueError):
                eng.norm(args.pop("x"), args.pop("weight"), args.pop("outputs"), **args)
        for eps in (-1.0, float("nan"), float("inf")):
            with pytest.raises(a2av.A2avError) as e:
                eng.norm(x, w, out, eps=eps)
            assert e.value.code == a2av.ERR_INVALID_ARG
        wide = [torch.empty(1, 16385, device="cuda")]
        with pytest.raises(a2av.A2avError) as e:
            eng.norm(wide, torch.ones(16385, device="cuda"), wide)
        assert e.value.code == a2av.ERR_UNSUPPORTED
        dw = torch.empty(64, device="cuda")
        with pytest.raises(a2av.A2avError):
            eng.norm_backward(x, w, x, out, d_weight=dw, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
        with pytest.raises(ValueError):
            eng.norm_backward(x, w, x, out, d_weight=dw, workspace=torch.empty(4096))
        with pytest.raises(ValueError):
            eng.norm_backward(x, w, [x[0][:2]], out)
        off = torch.empty(4 * packed[0].shape[1] + 8, dtype=torch.uint8, device="cuda")[8:].view(4, -1)
        with pytest.raises(a2av.A2avError) as e:
            eng.norm(x, w, [off], format="mxfp8")
        assert e.value.code == a2av.ERR_INVALID_ARG
        assert eng.status() == a2av.OK
