"""The norm, packed rows and the products on them where offsets pass 32 bits, where a
rank's tensors are missing or misaligned, and through the binding's own checks."""
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


@pytest.mark.parametrize("D", [8192, 8191])
def test_elements_beyond_32_bits(D):
    """2.2e9 elements in one buffer: the last rows are what they are in a buffer of their own."""
    R, tail = 270_000, 512
    x = torch.empty(R, D, dtype=torch.bfloat16, device="cuda")
    x[:-tail].fill_(1.0)
    x[-tail:].normal_()
    B = a2av.mx_row_bytes(D, "mxfp8")
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    with a2av.A2av(1) as eng:
        def run(t):
            n = t.shape[0]
            rows = torch.empty(n, B, dtype=torch.uint8, device="cuda")
            eng.quantise([t], [rows], "mxfp8")
            back = torch.empty_like(t)
            eng.dequantise([rows], [back], "mxfp8")
            y, packed = torch.empty_like(t), torch.empty_like(rows)
            eng.norm([t], w, [packed], format="mxfp8", plain=[y])
            d_x = torch.empty_like(t)
            eng.norm_backward([t], w, [back], [d_x])
            return [v[-tail:].clone() for v in (rows, back, y, packed, d_x)]
        whole, alone = run(x), run(x[-tail:].clone())
        assert eng.status() == a2av.OK
    assert all(torch.equal(a, b) for a, b in zip(whole, alone))


def test_product_of_rows_beyond_32_bits():
    """2.3 GB of packed rows, of three experts: the last one's results."""
    R, tail, D, N = 270_000, 700, 8192, 24
    B = a2av.mx_row_bytes(D, "mxfp8")
    rows = torch.zeros(R, B, dtype=torch.uint8, device="cuda")
    weights = torch.empty(3, N, B, dtype=torch.uint8, device="cuda")
    with a2av.A2av(1) as eng:
        eng.quantise([torch.randn(3 * N, D, device="cuda")], [weights.view(-1, B)], "mxfp8")
        eng.quantise([torch.randn(tail, D, device="cuda")], [rows[-tail:]], "mxfp8")
        counts = torch.tensor([[1000, R - tail - 1000, tail]], device="cuda")
        out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
        eng.expert_matmul_mx([rows], counts, [weights], [out], D, "mxfp8")
        alone = torch.empty(tail, N, dtype=torch.bfloat16, device="cuda")
        eng.expert_matmul_mx([rows[-tail:]], torch.tensor([[tail]], device="cuda"), [weights[2:]], [alone],
                             D, "mxfp8")
        assert eng.status() == a2av.OK
    assert torch.equal(out[-tail:], alone) and (out[:-tail] == 0).all()


def _calls(eng, t, none):
    """Every call on two ranks, the second without rows (`none`: its tensors are missing)."""
    H, fmt = 96, "mxfp4"
    B = a2av.mx_row_bytes(H, fmt)
    pair = lambda v: [v, None if none else v[:0].contiguous()]
    w, d_w = torch.linspace(1, 2, H, device="cuda"), torch.empty(H, device="cuda")
    new = lambda: torch.empty_like(t)
    s, y, d_x, rows, back = new(), new(), new(), torch.empty(t.shape[0], B, dtype=torch.uint8, device="cuda"), new()
    eng.norm(pair(t), w, pair(y), residual=pair(t), sums=pair(s))
    eng.norm(pair(t), w, pair(rows), format=fmt, plain=pair(new()))
    eng.norm_backward(pair(s), w, pair(t), pair(d_x), d_weight=d_w, d_sums=pair(y))
    eng.quantise(pair(t), pair(rows), fmt)
    eng.dequantise(pair(rows), pair(back), fmt)
    weights = rows[:8].view(1, 8, B).contiguous()
    out = torch.empty(t.shape[0], 8, dtype=t.dtype, device="cuda")
    counts = torch.tensor([[t.shape[0], 0], [0, 0]], device="cuda")
    eng.expert_matmul_mx(pair(rows), counts, [weights, weights], pair(out), H, fmt, activation="relu",
                         residual=pair(out.clone().zero_()))
    assert eng.status() == a2av.OK
    return [s, y, d_x, d_w, rows, back, out]


def test_missing_tensors_and_the_bindings_own_checks():
    t = torch.randn(40, 96, device="cuda").bfloat16()
    with a2av.A2av(2) as eng:
        want = _calls(eng, t, False)
        assert all(torch.equal(a, b) for a, b in zip(_calls(eng, t, True), want))
        eng._marshal = a2av._PlainMarshal
        assert all(torch.equal(a, b) for a, b in zip(_calls(eng, t, False), want))


@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
def test_weight_of_any_alignment(fmt):
    """The norm's weight four bytes off: the same values, whatever the row's own alignment."""
    for H, tokens in ((1024, 500), (1000, 3), (1001, 700), (7161, 2)):
        rng = np.random.default_rng(H)
        x = torch.from_numpy(rng.standard_normal((tokens, H))).cuda().bfloat16()
        w = torch.from_numpy(1 + 0.3 * rng.standard_normal(H)).float().cuda()
        off = torch.empty(H + 1, device="cuda")[1:].copy_(w)
        dy = torch.from_numpy(rng.standard_normal((tokens, H))).cuda().bfloat16()
        with a2av.A2av(1) as eng:
            for weight in (w, off):
                width = H if fmt is None else a2av.mx_row_bytes(H, fmt)
                out = torch.empty(tokens, width, dtype=x.dtype if fmt is None else torch.uint8, device="cuda")
                d_x, d_w = torch.empty_like(x), torch.empty(H, device="cuda")
                eng.norm([x], weight, [out], eps=1e-5, format=fmt)
                eng.norm_backward([x], weight, [dy], [d_x], d_weight=d_w, eps=1e-5)
                assert eng.status() == a2av.OK
                y = mx.norm(moe.f64(x), moe.f64(w), 1e-5)
                error = mx.norm_error(H)
                if fmt is None:
                    moe.close(out, y, error * np.abs(y), "bf16", "y")
                else:
                    v, scale = mx.unpack(out.cpu().numpy(), H, fmt)
                    rel, low = mx.HALF[fmt]
                    limit = np.maximum(rel * np.abs(y), low * scale) * (1 + error) + error * np.abs(y)
                    assert (np.abs(v - y) <= limit * (1 + 1e-9)).all()
                d, terms, size = mx.norm_backward(moe.f64(x), moe.f64(w), moe.f64(dy), 1e-5)
                moe.close(d_x, d, 4 * error * size, "bf16", "d_x")
                moe.close(d_w, terms.sum(0), (4 * error + (tokens + 8) * 2.0 ** -24) * np.abs(terms).sum(0),
                          "f32", "d_weight")


def test_two_graphs_with_a_workspace_each():
    """Two captured backward passes replayed on two streams at once."""
    H = 2048
    eng = a2av.A2av(1)
    w = torch.ones(H, device="cuda")
    s = [torch.randn(3000, H, device="cuda").bfloat16() for _ in range(2)]
    dy = [torch.randn_like(t) for t in s]
    want, got, graphs = [], [], []
    for a, b in zip(s, dy):
        d = torch.empty(H, device="cuda")
        eng.norm_backward([a], w, [b], [torch.empty_like(a)], d_weight=d)
        want.append(d)
    for a, b in zip(s, dy):
        d, d_x, graph = torch.empty(H, device="cuda"), torch.empty_like(a), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            eng.norm_backward([a], w, [b], [d_x], d_weight=d)
        got.append(d)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert eng.status() == a2av.OK
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    eng.close()
