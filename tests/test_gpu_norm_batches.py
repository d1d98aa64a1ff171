"""The norm and its gradients over batches of more rows than a GPU holds at once,
where rows are fetched ahead: by warps (up to 1024 features) and by blocks of 256 and
512 threads, across ranks of any number of rows; and called by two threads at once."""
import threading

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


def _rows(tokens, H, dtype, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    new = lambda t: torch.randn(t, H, device="cuda", generator=gen) * 2.0 ** torch.randint(
        -3, 4, (t, 1), device="cuda", generator=gen)
    return [new(t).to(moe.DTYPES[dtype]) for t in tokens]


def _weight(H):
    return 1 + 0.3 * torch.randn(H, device="cuda", generator=torch.Generator("cuda").manual_seed(9))


def _some(t):
    """Rows spread over a rank's, its first and last among them."""
    return np.unique(np.concatenate([np.arange(0, t, max(1, t // 40)), np.arange(min(t, 3)),
                                     np.arange(max(0, t - 3), t)])).astype(np.int64)


def _check_rows(got, y, fmt, dtype, what):
    H = y.shape[1]
    error = mx.norm_error(H)
    if fmt is None:
        return moe.close(got, y, error * np.abs(y), dtype, what)
    rows = got.cpu().numpy()
    V, B, _ = mx.layout(H, fmt)
    assert (rows[:, V + B:] == 0).all(), what
    v, scale = mx.unpack(rows, H, fmt)
    rel, low = mx.HALF[fmt]
    limit = np.maximum(rel * np.abs(y), low * scale) * (1 + error) + error * np.abs(y)
    assert (np.abs(v - y) <= limit * (1 + 1e-9)).all(), what
    top = np.abs(mx.blocks_of(y)).max(-1)
    s = 2.0 ** (rows[:, V:V + B].astype(np.float64) - 127)
    assert ((top * (1 + error) >= mx.MOST[fmt] * s / 2) | (s == 2.0 ** -127)).all(), what


def _forward(x, w, res, fmt, sums, plain=None):
    H = x[0].shape[1]
    width = H if fmt is None else a2av.mx_row_bytes(H, fmt)
    out = [torch.full((t.shape[0], width), 7, dtype=t.dtype if fmt is None else torch.uint8, device="cuda")
           for t in x]
    with a2av.A2av(len(x)) as eng:
        eng.norm(x, w, out, residual=res, sums=sums, eps=EPS, format=fmt, plain=plain)
        assert eng.status() == a2av.OK
    return out


def _backward(s, w, dy, ds, dx):
    dw = torch.full((s[0].shape[1],), 7.0, device="cuda")
    with a2av.A2av(len(s)) as eng:
        eng.norm_backward(s, w, dy, dx, d_weight=dw, d_sums=ds, eps=EPS)
        assert eng.status() == a2av.OK
    return dw


# (tokens of each rank, features, types): a warp a row, 128 and 512 threads a row
BATCHES = [([5003, 0, 4200, 7], 512, ("f32", "bf16", "f16")), ([1, 4301, 0, 5000], 1000, ("f32", "bf16", "f16")),
           ([0, 2600, 2501, 0], 1024, ("f32", "bf16", "f16")), ([3001, 0, 2700], 96, ("f32", "bf16", "f16")),
           ([1900, 0, 1801, 3], 4096, ("f32", "bf16", "f16")), ([300, 0, 201], 16384, ("bf16", "f16")),
           ([201, 1, 300], 12288, ("f32", "bf16")), ([700, 0, 301], 8192, ("f32",))]
CASES = [(tokens, H, dtype) for tokens, H, dtypes in BATCHES for dtype in dtypes]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm(case, fmt, residual):
    tokens, H, dtype = case
    x, w = _rows(tokens, H, dtype, 1), _weight(H)
    res = _rows(tokens, H, dtype, 2) if residual else None
    want = [(a.float() + b.float()).to(a.dtype) for a, b in zip(x, res)] if residual else x
    sums = [torch.full_like(t, 7) for t in x]
    plain = None if fmt is None else [torch.full_like(t, 7) for t in x]
    out = _forward(x, w, res, fmt, sums, plain)
    assert all(torch.equal(a, b) for a, b in zip(sums, want))
    for r, t in enumerate(tokens):
        at = torch.from_numpy(_some(t)).cuda()
        y = mx.norm(moe.f64(want[r][at]), moe.f64(w), EPS)
        _check_rows(out[r][at], y, fmt, dtype, f"rank {r}")
        if plain is not None:
            _check_rows(plain[r][at], y, None, dtype, f"rank {r}, plain")
        # (all rows, to what the types' roundings allow, in 64 bits on the device)
        s = want[r].double()
        all_y = s / (s.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
        if fmt is None:
            near = all_y.abs() * (moe.UNIT[dtype] * 1.01 + 2 * mx.norm_error(H)) + moe.TINY[dtype]
            assert ((out[r].double() - all_y).abs() <= near).all()
    # in place, and again: the same to the bit
    if residual:
        into = [t.clone() for t in res]
        again = _forward(x, w, into, fmt, into)
        assert all(torch.equal(a, b) for a, b in zip(again + into, out + want))
    else:
        assert all(torch.equal(a, b) for a, b in zip(_forward(x, w, None, fmt, None), out))


@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("case", [c for c in CASES if c[1] <= 4096], ids=str)
def test_rows_do_not_depend_on_their_batch(case, fmt):
    """All rows against calls on slices that are not fetched ahead."""
    tokens, H, dtype = case
    x, w, res = _rows(tokens, H, dtype, 3), _weight(H), _rows(tokens, H, dtype, 4)
    out = _forward(x, w, res, fmt, None)
    for r, t in enumerate(tokens):
        for i in range(0, t, 400):
            if H > 1024 and t - i < 400:
                continue  # (fewer rows than 2 an SM are summed by more threads)
            part = _forward([x[r][i:i + 400]], w, [res[r][i:i + 400]], fmt, None)[0]
            assert torch.equal(part, out[r][i:i + 400]), f"rank {r}, rows from {i}"


@pytest.mark.parametrize("more", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case, more):
    tokens, H, dtype = case
    s, w, dy = _rows(tokens, H, dtype, 5), _weight(H), _rows(tokens, H, dtype, 6)
    ds = _rows(tokens, H, dtype, 7) if more else None
    dx = [torch.full_like(t, 7) for t in s]
    dw = _backward(s, w, dy, ds, dx)
    error = 4 * mx.norm_error(H)
    terms, size = np.zeros(H), np.zeros(H)
    for r, t in enumerate(tokens):
        at = torch.from_numpy(_some(t)).cuda()
        d, _, mag = mx.norm_backward(moe.f64(s[r][at]), moe.f64(w), moe.f64(dy[r][at]), EPS)
        bound = error * mag
        if more:
            d = d + moe.f64(ds[r][at])
            bound = bound + 2.0 ** -24 * np.abs(d)
        moe.close(dx[r][at], d, bound, dtype, f"d_x of rank {r}")
        v = s[r].double()
        e = dy[r].double() * v / (v.square().mean(-1, keepdim=True) + EPS).sqrt()
        terms, size = terms + moe.f64(e.sum(0)), size + moe.f64(e.abs().sum(0))
    moe.close(dw, terms, (error + (sum(tokens) + 8) * 2.0 ** -24) * size, "f32", "d_weight")
    # over d_outputs, and over d_sums: the same to the bit
    for which in ("dy", "ds") if more else ("dy",):
        a, b = [t.clone() for t in dy], [t.clone() for t in ds] if more else None
        into = a if which == "dy" else b
        again = _backward(s, w, a, b, into)
        assert torch.equal(again, dw) and all(torch.equal(p, q) for p, q in zip(into, dx))


@pytest.mark.parametrize("backward", [False, True])
def test_two_threads(backward):
    """A handle and a stream each, rows of different width for the same kernel."""
    # 2048 and 8192 features of bf16: blocks of up to 256 threads (512: the gradients alike)
    widths, failed, results = (2048, 8192), [], {}
    data = {H: (_rows([4000], H, "bf16", 8), _weight(H), _rows([4000], H, "bf16", 10)) for H in widths}
    want = {}
    for H, (x, w, dy) in data.items():
        out = [torch.empty_like(x[0])]
        with a2av.A2av(1) as eng:
            if backward:
                eng.norm_backward(x, w, dy, out, eps=EPS)
            else:
                eng.norm(x, w, out, eps=EPS)
            assert eng.status() == a2av.OK
        want[H] = out[0]
    start = threading.Barrier(2)

    def work(H):
        x, w, dy = data[H]
        out = [torch.zeros_like(x[0])]
        stream = torch.cuda.Stream()
        try:
            with a2av.A2av(1) as eng:
                torch.cuda.synchronize()
                start.wait(60)
                for _ in range(1000):
                    if backward:
                        eng.norm_backward(x, w, dy, out, eps=EPS, stream=stream)
                    else:
                        eng.norm(x, w, out, eps=EPS, stream=stream)
                assert eng.status(stream) == a2av.OK
            results[H] = out[0]
        except Exception as e:
            failed.append((H, e))

    threads = [threading.Thread(target=work, args=(H,)) for H in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert all(torch.equal(results[H], want[H]) for H in widths)
