"""Packed rows on the GPU: codes, scales and bytes against the definition, to the
bit, and back."""
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


def _place(values, dt, offset=0):
    buf = torch.empty(values.size + offset, dtype=dt, device="cuda")
    view = buf[offset:].view(values.shape)
    view.copy_(torch.from_numpy(np.ascontiguousarray(values)))
    return view


def _values(rows, D, seed):
    """Blocks of very different size, and some of zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, D))
    size = 2.0 ** rng.integers(-12, 10, (rows, -(-D // 32))) * (rng.random((rows, -(-D // 32))) > 0.1)
    return x * size.repeat(32, 1)[:, :D]


def _quantise(x, fmt, stream=None):
    D = x[0].shape[1]
    rows = [torch.full((t.shape[0], a2av.mx_row_bytes(D, fmt)), 7, dtype=torch.uint8, device="cuda") for t in x]
    with a2av.A2av(len(x)) as eng:
        eng.quantise(x, rows, fmt, stream=stream)
        assert eng.status(stream) == a2av.OK
    return rows


def _dequantise(rows, D, dt, fmt, offset=0):
    out = [_place(np.full((t.shape[0], D), 7.0), dt, offset) for t in rows]
    with a2av.A2av(len(rows)) as eng:
        eng.dequantise(rows, out, fmt)
        assert eng.status() == a2av.OK
    return out


SHAPES = [([1], 1), ([2, 0, 3], 31), ([5], 32), ([40], 33), ([7], 64), ([3], 100), ([300], 256), ([9], 1000),
          ([8], 1001), ([64, 65], 2048), ([4] * 8, 7168), ([0], 32), ([2], 20000)]


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_there_and_back(shape, dtype, fmt):
    tokens, D = shape
    x = [_place(_values(t, D, r), moe.DTYPES[dtype]) for r, t in enumerate(tokens)]
    rows = _quantise(x, fmt)
    back = _dequantise(rows, D, moe.DTYPES[dtype], fmt)
    for r, t in enumerate(tokens):
        want = mx.pack(moe.f64(x[r]), fmt)
        assert np.array_equal(rows[r].cpu().numpy(), want), f"rank {r}"
        values = torch.from_numpy(mx.unpack(want, D, fmt)[0]).to(moe.DTYPES[dtype])
        assert torch.equal(back[r].cpu(), values), f"rank {r}"


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("offset", [1, 4])
def test_unaligned_values(offset, fmt):
    for D in (64, 2048):
        x = [_place(_values(11, D, 3), torch.float16, offset)]
        rows = _quantise(x, fmt)
        want = mx.pack(moe.f64(x[0]), fmt)
        assert np.array_equal(rows[0].cpu().numpy(), want)
        back = _dequantise(rows, D, torch.float16, fmt, offset)[0]
        assert torch.equal(back.cpu(), torch.from_numpy(mx.unpack(want, D, fmt)[0]).half())


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_special_values(fmt):
    """Every code and midpoint, the largest and smallest magnitudes, zeros of both signs;
    a NaN or an infinity takes its block with it and no other."""
    t = mx.TABLE[fmt]
    near = np.concatenate([t, (t[1:] + t[:-1]) / 2, np.nextafter(np.float32(t), np.float32(9e9)).clip(0, t[-1])])
    near = np.concatenate([near, -near])
    near = np.concatenate([near, np.zeros(-len(near) % 31)]).reshape(-1, 31)
    x = np.concatenate([near, np.full((len(near), 1), t[-1])], 1).reshape(1, -1)  # (scales of 1)
    special = np.zeros((14, 32))
    special[0, 3] = np.nan
    special[1, 31] = np.inf
    special[2, 0] = -np.inf
    special[3] = 3.4e38
    special[4] = 1e-45
    special[5, :2] = 2.0 ** -126, 2.0 ** -149
    special[6] = -0.0
    special[7, 4] = 1.0
    special[8, :2] = t[-1], np.nextafter(np.float32(t[-1]), np.float32(9e9))
    special[9, 0] = np.nextafter(np.float32(t[-1] * 2.0 ** -30), np.float32(1))
    special[10, 0] = t[-1] * 2.0 ** -127
    special[11, 0] = np.nextafter(np.float32(t[-1] * 2.0 ** -127), np.float32(1))
    special[12, 5] = 2.0 ** 127
    x = np.float32(np.concatenate([x, special.reshape(1, -1)], 1))
    for width in (x.shape[1], 32 * 5 + 31):  # vectors, and none
        part = x[:, -width:] if width % 4 == 0 else x[:, :width]
        rows = _quantise([_place(part, torch.float32)], fmt)
        want = mx.pack(part.astype(np.float64), fmt)
        assert np.array_equal(rows[0].cpu().numpy(), want)
        back = _dequantise(rows, part.shape[1], torch.float32, fmt)[0].cpu().numpy()
        ref = np.float32(mx.unpack(want, part.shape[1], fmt)[0])
        assert np.array_equal(back, ref, equal_nan=True)


def test_every_byte_of_a_packed_row_means_what_it_says():
    """All 256 codes under all 256 scales, 8 bits; all pairs of 4-bit codes."""
    for fmt, per in (("mxfp8", 32), ("mxfp4", 16)):
        codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
        if fmt == "mxfp8":
            codes[codes % 128 == 127] = 0  # (NaN codes: below)
        scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 256 // per, 1)
        D = 256 * 32 // per
        rows = np.zeros((256, mx.layout(D, fmt)[2]), np.uint8)
        rows[:, :256], rows[:, 256:256 + scales.shape[1]] = codes, scales
        back = _dequantise([torch.from_numpy(rows).cuda()], D, torch.float32, fmt)[0].cpu().numpy()
        with np.errstate(over="ignore"):
            want = np.float32(mx.unpack(rows, D, fmt)[0])
        assert np.array_equal(back, want, equal_nan=True)
    rows = np.zeros((1, 64), np.uint8)
    rows[0, :3], rows[0, 32] = (0x7f, 0xff, 0x38), 127
    back = _dequantise([torch.from_numpy(rows).cuda()], 32, torch.float32, "mxfp8")[0][0]
    assert back[:2].isnan().all() and back[2] == 1


@pytest.mark.parametrize("D", [64, 101])
def test_received_rows_alone(D):
    """With a dispatch's splits: rows past the received ones are left as they were, also where the
    counts change between a graph's replays; splits that do not fit write nothing."""
    W, held = 3, (40, 7, 0)
    x = [_place(_values(n, D, 7 + p), torch.bfloat16) for p, n in enumerate(held)]
    whole = _quantise(x, "mxfp8")
    back = _dequantise(whole, D, torch.bfloat16, "mxfp8")
    splits = torch.tensor([[5, 0, 0], [0, 7, 0], [21, 0, 0]], device="cuda")
    rows, out = [torch.full_like(t, 9) for t in whole], [torch.full_like(t, 9) for t in x]
    with a2av.A2av(W) as eng:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            eng.quantise(x, rows, "mxfp8", in_splits=splits)
            eng.dequantise(rows, out, "mxfp8", in_splits=splits)
        for S in ([[5, 0, 0], [0, 7, 0], [21, 0, 0]], [[0, 0, 0], [0, 0, 0], [0, 0, 0]],
                  [[40, 1, 0], [0, 2, 0], [0, 3, 0]]):
            splits.copy_(torch.tensor(S))
            for t in rows + out:
                t.fill_(9)
            graph.replay()
            assert eng.status() == a2av.OK
            for p in range(W):
                n = sum(S[r][p] for r in range(W))
                assert torch.equal(rows[p][:n], whole[p][:n]) and (rows[p][n:] == 9).all()
                assert torch.equal(out[p][:n], back[p][:n]) and (out[p][n:] == 9).all()
        for S in ([[41, 0, 0]] + [[0] * 3] * 2, [[-1, 0, 0], [5, 0, 0], [0] * 3], [[0, 0, 1]] + [[0] * 3] * 2,
                  [[2 ** 62, 0, 0], [2 ** 62, 0, 0], [2 ** 62, 0, 0]]):
            splits.copy_(torch.tensor(S))
            for t in rows + out:
                t.fill_(9)
            eng.quantise(x, rows, "mxfp8", in_splits=splits)
            assert eng.status() == a2av.ERR_BAD_SPLITS
            eng.dequantise(whole, out, "mxfp8", in_splits=splits)
            assert eng.status() == a2av.ERR_BAD_SPLITS
            assert all((t == 9).all() for t in rows + out)
        with pytest.raises(ValueError):
            eng.quantise(x, rows, "mxfp8", in_splits=splits.int())


def test_graph_and_streams():
    x = [_place(_values(50, 512, 5), torch.bfloat16), _place(_values(7, 512, 6), torch.bfloat16)]
    want = _quantise(x, "mxfp4")
    rows, out = [torch.zeros_like(t) for t in want], [torch.zeros_like(t) for t in x]
    back = _dequantise(want, 512, torch.bfloat16, "mxfp4")
    side = torch.cuda.Stream()
    with a2av.A2av(2) as eng:
        side.wait_stream(torch.cuda.current_stream())
        eng.quantise(x, rows, "mxfp4", stream=side)
        eng.dequantise(rows, out, "mxfp4", stream=side)
        assert eng.status(side) == a2av.OK
        assert all(torch.equal(a, b) for a, b in zip(rows + out, want + back))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            eng.quantise(x, rows, "mxfp4")
            eng.dequantise(rows, out, "mxfp4")
        for t in rows + out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(rows + out, want + back))
        there, again = eng.bind_quantise(x, rows, "mxfp4"), eng.bind_dequantise(rows, out, "mxfp4")
        for t in x:
            t.neg_()
        there()
        again()
        assert eng.status() == a2av.OK
        assert all(torch.equal(a, -b) for a, b in zip(out, back))


def test_refusals():
    x = [torch.zeros(4, 64, device="cuda")]
    rows = [torch.empty(4, a2av.mx_row_bytes(64, "mxfp8"), dtype=torch.uint8, device="cuda")]
    with a2av.A2av(1) as eng:
        for call in (eng.quantise, eng.dequantise):
            back = call == eng.dequantise
            for a, b, fmt in ((x, rows, "mxfp4"), (x, rows, None), (x, rows, "int8"), (x, [rows[0][:3]], "mxfp8"),
                              ([x[0].double()], rows, "mxfp8"), ([x[0].long()], rows, "mxfp8"),
                              (x, [rows[0].char()], "mxfp8"), ([x[0].cpu()], rows, "mxfp8"), (x + x, rows, "mxfp8"),
                              ([x[0].t()], rows, "mxfp8"), (x, [None], "mxfp8")):
                with pytest.raises(ValueError):
                    call(*((b, a) if back else (a, b)), fmt)
            n = rows[0].numel()
            off = [torch.empty(n + 8, dtype=torch.uint8, device="cuda")[8:].view(4, -1)]
            with pytest.raises(a2av.A2avError) as e:
                call(*((off, x) if back else (x, off)), "mxfp8")
            assert e.value.code == a2av.ERR_INVALID_ARG
        assert eng.status() == a2av.OK
