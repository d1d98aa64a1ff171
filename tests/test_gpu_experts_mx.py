"""The experts' products on packed rows and weights, on the GPU: results against
the definition in 64 bits on the values that the packed rows stand for, with error
bounds from the arithmetic, and what they refuse."""
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


def _counts(rng, W, K, rows, kind):
    """Items of each (rank, expert): `rows` a group on average."""
    c = rng.integers(0, 2 * rows + 1, (W, W * K))
    if kind == "empty":
        c[:] = 0
    if kind == "one":
        c[:] = 0
        c[rng.integers(W), rng.integers(W * K)] = rows
    if kind == "sparse":
        c = c * (rng.random(c.shape) < 0.4)
    return c.astype(np.int64)


def _packed(rng, rows, D, fmt, std):
    """Packed rows of random codes and scales (whose blocks differ up to 2^4 in size),
    and the values that they stand for."""
    V, B, size = mx.layout(D, fmt)
    x = rng.standard_normal((rows, D)).astype(np.float32) * std
    x *= (2.0 ** rng.integers(-2, 3, (rows, B))).repeat(32, 1)[:, :D]
    t = torch.from_numpy(x).cuda()
    out = torch.empty(rows, size, dtype=torch.uint8, device="cuda")
    with a2av.A2av(1) as eng:  # (tested by itself)
        eng.quantise([t], [out], fmt)
        assert eng.status() == a2av.OK
    return out, mx.unpack(out.cpu().numpy(), D, fmt)[0]


def _case(W, K, D, N, rows, dtype, fmt, gated, kind="random", seed=0, offset=0, slack=0):
    rng = np.random.default_rng(seed)
    dt = moe.DTYPES[dtype]
    counts = _counts(rng, W, K, rows, kind)
    Z = 2 * N if gated else N
    held = [int(counts[:, p * K:(p + 1) * K].sum()) + slack for p in range(W)]

    def place(values):
        buf = torch.empty(values.size + offset, dtype=dt, device="cuda")
        view = buf[offset:].view(values.shape)
        view.copy_(torch.from_numpy(np.ascontiguousarray(values)))
        return view

    x = [_packed(rng, m, D, fmt, 1.0) for m in held]
    w = [_packed(rng, K * Z, D, fmt, D ** -0.5) for _ in range(W)]
    return {"W": W, "K": K, "D": D, "N": N, "Z": Z, "counts": counts, "held": held, "dtype": dtype,
            "fmt": fmt, "gated": gated, "place": place, "d_counts": torch.from_numpy(counts).cuda(),
            "x": [a for a, _ in x], "x64": [b for _, b in x],
            "w": [a.view(K, Z, -1) for a, _ in w], "w64": [b.reshape(K, Z, D) for _, b in w],
            "b": [place(rng.standard_normal((K, Z)) * 0.3) for _ in range(W)],
            "res": [place(rng.standard_normal((m, N))) for m in held],
            "owner": [moe.row_experts(counts, p, K) for p in range(W)]}


def _run(c, name, bias, residual, stream=None, x=None, eng=None, out=None):
    out = out or [c["place"](np.full((m, c["N"]), 7.0)) for m in c["held"]]
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    own = eng or a2av.A2av(c["W"])
    own.expert_matmul_mx(x or c["x"], c["d_counts"], c["w"], out, c["D"], c["fmt"], activation=name,
                         gated=c["gated"], bias=c["b"] if bias else None,
                         residual=c["res"] if residual else None, stream=stream)
    assert own.status(stream) == a2av.OK
    if eng is None:
        own.close()
    return out


def _check(c, name, bias, residual, out):
    for p in range(c["W"]):
        n = c["owner"][p].size
        y, _, bound, _ = moe.expert_forward(
            c["x64"][p][:n], c["owner"][p], c["w64"][p], moe.f64(c["b"][p]) if bias else None,
            moe.f64(c["res"][p])[:n] if residual else None, name, c["gated"])
        bound = bound + 2.0 ** -23 * np.abs(y)
        moe.close(out[p][:n], y, bound, c["dtype"], f"peer {p}")
        assert (out[p][n:] == 7).all(), "rows past the groups written"


# (W, K, D, N, rows of a group on average)
SHAPES = [(1, 1, 32, 8, 1), (1, 1, 64, 128, 1), (1, 1, 256, 128, 300), (2, 3, 128, 72, 20),
          (1, 4, 200, 264, 70), (4, 2, 96, 40, 9), (1, 1, 8, 8, 5), (1, 2, 1000, 136, 129),
          (2, 2, 320, 512, 40), (1, 1, 33, 17, 50), (2, 2, 65, 64, 30), (1, 3, 64, 63, 10),
          (8, 8, 64, 64, 3), (1, 1, 2048, 256, 2), (1, 2, 544, 300, 240), (1, 1, 1, 1, 1),
          (2, 1, 4096, 130, 70), (1, 1, 288, 256, 700)]
EPILOGUES = [("none", False, False, False), ("silu", True, False, False), ("gelu", False, True, True),
             ("relu", False, True, False), ("silu", False, False, True), ("gelu", True, True, True),
             ("none", True, True, False), ("none", False, False, True)]


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("epilogue", EPILOGUES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_product(shape, epilogue, fmt):
    name, gated, bias, residual = epilogue
    dtype = "bf16" if (shape[3] + len(name)) % 2 else "f16"
    c = _case(*shape, dtype, fmt, gated, seed=1, slack=3)
    _check(c, name, bias, residual, _run(c, name, bias, residual))


@pytest.mark.parametrize("kind", ["empty", "one", "sparse"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_uneven_groups(fmt, gated, kind):
    c = _case(3, 4, 96, 80, 150, "bf16", fmt, gated, kind, seed=2, slack=1)
    _check(c, "silu", True, False, _run(c, "silu", True, False))


@pytest.mark.parametrize("offset", [1, 4])
def test_unaligned_results(offset):
    c = _case(2, 2, 128, 64, 33, "f16", "mxfp4", True, seed=3, offset=offset)
    _check(c, "silu", True, True, _run(c, "silu", True, True))


def test_many_groups():
    """More groups than a block's table has entries: 32 ranks, 32 experts each."""
    c = _case(32, 32, 32, 16, 1, "bf16", "mxfp8", False, "sparse", seed=4)
    _check(c, "none", False, False, _run(c, "none", False, False))


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_blocks_of_nan_stay_within_their_rows(fmt):
    """NaN scales in rows of one group, and in the slack past the groups, reach no other row."""
    c = _case(1, 3, 128, 64, 40, "bf16", fmt, False, "random", seed=5, slack=2)
    n = c["owner"][0].size
    clean = _run(c, "none", True, False)
    x = c["x"][0].clone()
    x[n:] = 255
    bad = torch.from_numpy(np.nonzero(c["owner"][0] == 1)[0]).cuda()
    x[bad, mx.layout(128, fmt)[0] + 2] = 255
    out = _run(c, "none", True, False, x=[x])
    other = torch.from_numpy(np.nonzero(c["owner"][0] != 1)[0]).cuda()
    assert torch.equal(out[0][other], clean[0][other])
    assert out[0][bad].isnan().all()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_scales_far_apart(fmt):
    """Blocks whose scales are 2^100 apart on one side and as far the other way on the other."""
    rng = np.random.default_rng(6)
    D, N, M = 64, 32, 20
    c = _case(1, 1, D, N, M, "bf16", fmt, False, "one", seed=6)
    V = mx.layout(D, fmt)[0]
    for t, by in ((c["x"][0], 50), (c["w"][0], -50)):
        t[..., V] += by % 256  # (bytes wrap around)
        t[..., V + 1] += -by % 256
    n = c["owner"][0].size
    c["x64"] = [mx.unpack(c["x"][0].cpu().numpy(), D, fmt)[0]]
    c["w64"] = [mx.unpack(c["w"][0].cpu().numpy().reshape(N, -1), D, fmt)[0].reshape(1, N, D)]
    assert n == M and np.abs(c["x64"][0]).max() > 1e10 and np.abs(c["w64"][0]).max() > 1e10
    _check(c, "none", False, False, _run(c, "none", False, False))


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_repeated_graph_and_streams(fmt):
    """The same to the bit: again, on a side stream, in a graph, bound; new counts on replay."""
    c = _case(2, 3, 512, 264, 90, "bf16", fmt, True, seed=7)
    want = _run(c, "silu", True, False)
    _check(c, "silu", True, False, want)
    assert all(torch.equal(a, b) for a, b in zip(_run(c, "silu", True, False), want))
    assert all(torch.equal(a, b) for a, b in zip(_run(c, "silu", True, False, stream=torch.cuda.Stream()), want))
    out = [torch.zeros_like(t) for t in want]
    with a2av.A2av(2) as eng:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            eng.expert_matmul_mx(c["x"], c["d_counts"], c["w"], out, c["D"], fmt, activation="silu",
                                 gated=True, bias=c["b"])
        graph.replay()
        assert eng.status() == a2av.OK
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        fewer = c["d_counts"].clone()
        fewer[0, 0] = 0
        kept = c["d_counts"].clone()
        c["d_counts"].copy_(fewer)
        graph.replay()
        assert eng.status() == a2av.OK
        c["counts"] = fewer.cpu().numpy()
        c["owner"] = [moe.row_experts(c["counts"], p, 3) for p in range(2)]
        for p in range(2):
            out[p][c["owner"][p].size:] = 7
        _check(c, "silu", True, False, out)
        c["d_counts"].copy_(kept)
        call = eng.bind_expert_matmul_mx(c["x"], c["d_counts"], c["w"], out, c["D"], fmt, activation="silu",
                                         gated=True, bias=c["b"])
        call()
        assert eng.status() == a2av.OK
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_calls_at_once():
    """On two streams of one handle."""
    a = _case(1, 4, 1024, 512, 100, "bf16", "mxfp8", False, seed=8)
    b = _case(1, 2, 2048, 256, 30, "bf16", "mxfp4", True, seed=9)
    want = _run(a, "gelu", True, False), _run(b, "silu", False, False)
    outs = [torch.empty_like(want[0][0])], [torch.empty_like(want[1][0])]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with a2av.A2av(1) as eng:
        for _ in range(5):
            eng.expert_matmul_mx(a["x"], a["d_counts"], a["w"], outs[0], a["D"], "mxfp8", activation="gelu",
                                 bias=a["b"], stream=streams[0])
            eng.expert_matmul_mx(b["x"], b["d_counts"], b["w"], outs[1], b["D"], "mxfp4", activation="silu",
                                 gated=True, stream=streams[1])
        torch.cuda.synchronize()
        assert eng.status() == a2av.OK
    assert torch.equal(outs[0][0], want[0][0]) and torch.equal(outs[1][0], want[1][0])


def test_bad_counts_write_nothing():
    c = _case(2, 2, 64, 64, 10, "bf16", "mxfp8", False, seed=10)
    for value in (-1, 10 ** 6, 1 << 40):
        counts = c["d_counts"].clone()
        counts[1, 2] = value
        out = [torch.full_like(t, 7) for t in c["res"]]
        with a2av.A2av(2) as eng:
            eng.expert_matmul_mx(c["x"], counts, c["w"], out, 64, "mxfp8")
            assert eng.status() == a2av.ERR_BAD_SPLITS
        assert all((t == 7).all() for t in out)


def test_refusals():
    c = _case(1, 2, 64, 64, 10, "bf16", "mxfp8", False, seed=11)
    x, w, counts, out = c["x"], c["w"], c["d_counts"], [torch.empty_like(t) for t in c["res"]]
    with a2av.A2av(1) as eng:
        for bad in (dict(rows=[x[0][:3]]), dict(rows=[x[0].char()]), dict(weights=[w[0][:, :5]]),
                    dict(weights=[w[0].view(-1, w[0].shape[2])]), dict(outputs=[out[0].float()]),
                    dict(in_features=96), dict(in_features=0), dict(format="mxfp4"), dict(format=None),
                    dict(activation="tanh"), dict(bias=c["res"]), dict(residual=[out[0].half()]),
                    dict(counts=counts.int()), dict(gated=True)):
            args = {"rows": x, "counts": counts, "weights": w, "outputs": out, "in_features": 64,
                    "format": "mxfp8", **bad}
            with pytest.raises(ValueError):
                eng.expert_matmul_mx(**args)
        off = torch.empty(x[0].numel() + 8, dtype=torch.uint8, device="cuda")[8:].view(x[0].shape)
        with pytest.raises(a2av.A2avError) as e:
            eng.expert_matmul_mx([off], counts, w, out, 64, "mxfp8")
        assert e.value.code == a2av.ERR_INVALID_ARG
        assert eng.status() == a2av.OK
