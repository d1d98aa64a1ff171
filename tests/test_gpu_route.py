"""The router on the GPU: keys, weights, counts and gradients against the
definition in 64 bits, and what it refuses."""
import ctypes

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


# (tokens of each rank, E, k, score, bias, groups, top_groups, group_top, renormalise)
CASES = [
    ([1], 1, 1, "softmax", False, 1, 1, 1, True),
    ([1], 64, 2, "softmax", False, 1, 1, 1, True),
    ([3, 0, 5, 1], 64, 2, "softmax", False, 1, 1, 1, False),
    ([40, 33], 37, 5, "softmax", False, 1, 1, 1, True),
    ([17, 64, 1], 30, 30, "softmax", False, 1, 1, 1, False),
    ([100, 3], 256, 8, "sigmoid", True, 8, 4, 2, True),
    ([9, 70], 256, 8, "sigmoid", True, 8, 4, 2, False),
    ([55], 60, 6, "sigmoid", False, 4, 2, 1, True),
    ([31, 31], 160, 6, "softmax", False, 8, 3, 1, False),
    ([12], 96, 7, "softmax", False, 32, 9, 1, True),
    ([300, 0], 128, 1, "sigmoid", False, 1, 1, 1, False),
    ([25], 1024, 32, "softmax", False, 1, 1, 1, True),
    ([10, 11], 999, 9, "sigmoid", True, 3, 2, 2, True),
    ([700], 24, 3, "sigmoid", True, 6, 6, 1, True),
    ([19], 512, 16, "sigmoid", False, 16, 5, 2, False),
    ([14], 33, 4, "softmax", False, 11, 3, 1, False),
    # tokens enough for a thread a token
    ([2100], 64, 2, "softmax", False, 1, 1, 1, True),
    ([1500, 0, 700], 256, 8, "sigmoid", True, 8, 4, 2, True),
    ([2049], 24, 3, "softmax", False, 6, 2, 1, False),
    ([1100, 1000], 128, 1, "sigmoid", False, 1, 1, 1, False),
    ([33, 2200], 160, 7, "softmax", False, 5, 3, 1, False),
    ([2300], 8, 8, "sigmoid", True, 2, 2, 2, True),
]


def _logits(rng, n, E, dtype, kind):
    x = rng.standard_normal((n, E)) * 2
    if kind == "ties":  # few distinct values: the lowest index has to win
        x = np.round(x)
    elif kind == "masked":
        x[rng.random((n, E)) < 0.5] = -np.inf
        if n > 2:
            x[1] = -np.inf
    elif kind == "lowest":  # the type's lowest value in masked places
        x[rng.random((n, E)) < 0.5] = torch.finfo(moe.DTYPES[dtype]).min
    return torch.from_numpy(x).to(moe.DTYPES[dtype])


def _choice(x32, case, bias):
    """Choices with the 32-bit arithmetic the definition names (torch on the GPU)."""
    _, _, _, score, _, _, _, group_top, _ = case
    if score == "softmax" and bias is None and group_top == 1:
        return x32.cpu().numpy()
    assert score == "sigmoid"
    c = 1 / (1 + torch.exp(-x32))
    return (c if bias is None else c + bias).cpu().numpy()


def _run(case, dtype, kind, seed, stream=None, scale=1.5):
    T, E, k, score, with_bias, groups, top_groups, group_top, renorm = case
    rng = np.random.default_rng(seed)
    W = len(T)
    x = [_logits(rng, n, E, dtype, kind).cuda() for n in T]
    bias = torch.from_numpy(rng.standard_normal(E).astype(np.float32) * 0.1).cuda() if with_bias else None
    keys = [torch.full((n, k), -7, dtype=torch.int32, device="cuda") for n in T]
    w = [torch.full((n, k), -7.0, device="cuda") for n in T]
    counts = torch.full((W, E), -7, dtype=torch.int64, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    with a2av.A2av(W) as eng:
        eng.route(x, keys, w, k, counts=counts, bias=bias, score=score, groups=groups,
                  top_groups=top_groups, group_top=group_top, renormalise=renorm, scale=scale,
                  stream=stream)
        assert eng.status(stream) == a2av.OK
    return x, bias, keys, w, counts


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "lowest"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_route(case, kind, dtype):
    T, E, k, score, _, groups, top_groups, group_top, renorm = case
    x, bias, keys, w, counts = _run(case, dtype, kind, 5)
    for r, n in enumerate(T):
        c = _choice(x[r].float(), case, bias)
        x64 = moe.f64(x[r])
        ids = np.stack([moe.choose(row, k, groups, top_groups, group_top) for row in c]) if n else \
            np.zeros((0, k), int)
        assert np.array_equal(keys[r].cpu().numpy(), ids)
        ref = np.stack([moe.weights_of(x64[t], ids[t], score, renorm, 1.5) for t in range(n)]) if n else \
            np.zeros((0, k))
        # exp of a rounded difference (|x| 2^-24) and its own 2 ulp, twice; a sum of E; two divisions
        with np.errstate(invalid="ignore"):
            big = np.where(np.isfinite(x64), np.abs(x64), 0).max(initial=0) if kind != "lowest" else 16
        bound = np.abs(ref) * 2.0 ** -24 * (4 * min(big, 90) + E + 16) + 2.0 ** -126
        moe.close(w[r], ref, bound, "f32", f"weights of rank {r}")
        assert np.array_equal(counts[r].cpu().numpy(), np.bincount(ids.reshape(-1), minlength=E))


def test_softmax_with_bias_chooses_by_probability():
    """Bias added to probabilities: the keys must be the top k up to the scores' rounding."""
    T, E, k = 200, 48, 4
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    bias = torch.from_numpy(rng.standard_normal(E).astype(np.float32) * 0.02).cuda()
    keys = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    with a2av.A2av(1) as eng:
        eng.route([x], [keys], [w], k, bias=bias, groups=4, top_groups=2, group_top=2,
                  renormalise=False)
        assert eng.status() == a2av.OK
    got = keys.cpu().numpy()
    for t in range(T):
        p = moe.scores(moe.f64(x[t]), "softmax")
        c = p + moe.f64(bias)
        g = np.sort(c.reshape(4, 12), axis=1)[:, -2:].sum(axis=1)
        assert len(set(got[t])) == k
        groups = sorted(set(got[t] // 12))
        assert len(groups) <= 2
        assert all(g[i] >= np.sort(g)[-2] - 1e-5 for i in groups)
        chosen = c[got[t]]
        assert np.all(np.diff(chosen) <= 1e-6)
        moe.close(w[t], p[got[t]], np.abs(p[got[t]]) * 2.0 ** -17, "f32", "weights")


def test_nan_is_chosen_last_and_keys_stay_valid():
    x = torch.randn((6, 8), device="cuda")
    x[0, 3] = float("nan")
    x[1] = float("nan")
    x[2, :] = float("inf")
    keys = torch.empty((6, 3), dtype=torch.int32, device="cuda")
    w = torch.empty((6, 3), device="cuda")
    counts = torch.empty((1, 8), dtype=torch.int64, device="cuda")
    with a2av.A2av(1) as eng:
        eng.route([x], [keys], [w], 3, counts=counts, score="sigmoid")
        assert eng.status() == a2av.OK
    k = keys.cpu().numpy()
    assert 3 not in k[0]
    assert k[1].tolist() == [0, 1, 2] and k[2].tolist() == [0, 1, 2]
    assert torch.isnan(w[1]).all() and torch.isfinite(w[0]).all()
    assert int(counts.sum()) == 18


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["normal", "masked"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_route_backward(case, kind, dtype):
    T, E, k, score, _, groups, top_groups, group_top, renorm = case
    x, bias, keys, w, _ = _run(case, dtype, kind, 9)
    g = [torch.randn((n, k), device="cuda") for n in T]
    d = [torch.full_like(a, 7.0) for a in x]
    with a2av.A2av(len(T)) as eng:
        eng.route_backward(x, keys, g, d, k, score=score, renormalise=renorm, scale=1.5)
        assert eng.status() == a2av.OK
    for r, n in enumerate(T):
        x64, g64, ids = moe.f64(x[r]), moe.f64(g[r]), keys[r].cpu().numpy()
        for t in range(n):
            ref = moe.weights_gradient(x64[t], ids[t], g64[t], score, renorm, 1.5)
            # the gradient is a difference: its error goes by the largest g * s
            s = moe.scores(x64[t], score)
            if renorm and score == "softmax":
                s = s * 0
                s[ids[t]] = moe.scores(x64[t][ids[t]], score)
            top = s[ids[t]]
            scale = 1.5 * np.abs(g64[t]).max() * (1 if not renorm or score == "softmax" else
                                                  1 / max(top.sum(), 1e-30))
            bound = 2.0 ** -24 * (E + 64) * 8 * scale * np.maximum(s, top.max() * s)
            moe.close(d[r][t], ref, bound, dtype, f"gradient of rank {r} token {t}")


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                          ("sigmoid", True)])
def test_gradient_formula_against_differences(score, renorm):
    """The definition's gradient against central differences of its weights (64 bits)."""
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal(12), rng.standard_normal(4)
    ids = moe.choose(x, 4, 1, 1, 1)
    d = moe.weights_gradient(x, ids, g, score, renorm, 2.0)
    h = 1e-5
    for i in range(12):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        num = ((moe.weights_of(a, ids, score, renorm, 2.0) - moe.weights_of(b, ids, score, renorm, 2.0)) * g).sum() / (2 * h)
        assert abs(num - d[i]) < 1e-8


def test_streams_and_unaligned_rows():
    """Another stream than the tensors' own, and rows that start at any element."""
    base = torch.randn(70 * 64 + 1, device="cuda").bfloat16()
    x = base[1:].view(70, 64)
    outs = []
    for stream in (None, torch.cuda.Stream()):
        keys = torch.empty((70, 4), dtype=torch.int32, device="cuda")
        w = torch.empty((70, 4), device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        with a2av.A2av(1) as eng:
            eng.route([x], [keys], [w], 4, stream=stream)
            assert eng.status(stream) == a2av.OK
        outs.append((keys.cpu(), w.cpu()))
    ref = x.float().sort(dim=-1, descending=True, stable=True).indices[:, :4].int().cpu()
    for k, w in outs:
        assert torch.equal(k, ref)
    assert torch.equal(outs[0][1], outs[1][1])


def test_bound_call_and_graph():
    x = torch.randn((16, 64), device="cuda")
    keys = torch.empty((16, 2), dtype=torch.int32, device="cuda")
    w = torch.empty((16, 2), device="cuda")
    counts = torch.empty((1, 64), dtype=torch.int64, device="cuda")
    with a2av.A2av(1) as eng:
        call = eng.bind_route([x], [keys], [w], 2, counts=counts)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(torch.cuda.current_stream())
        for _ in range(3):
            x.copy_(torch.randn((16, 64), device="cuda"))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(keys.cpu(), x.sort(descending=True, stable=True).indices[:, :2].int().cpu())
            assert int(counts.sum()) == 32


def test_bad_keys_in_backward():
    x = torch.randn((4, 8), device="cuda")
    keys = torch.tensor([[0, 1], [8, 1], [-1, 2], [3, 4]], dtype=torch.int32, device="cuda")
    g, d = torch.ones((4, 2), device="cuda"), torch.full((4, 8), 7.0, device="cuda")
    with a2av.A2av(1) as eng:
        eng.route_backward([x], [keys], [g], [d], 2, score="sigmoid", renormalise=False)
        assert eng.status() == a2av.ERR_BAD_INDEX
        assert eng.status() == a2av.OK
    assert d[1].abs().sum() == 0 and d[2].abs().sum() == 0 and d[3].abs().sum() > 0


def test_refusals():
    x = torch.randn((4, 8), device="cuda")
    keys = torch.empty((4, 2), dtype=torch.int32, device="cuda")
    w = torch.empty((4, 2), device="cuda")
    with a2av.A2av(1) as eng:
        for kw in (dict(groups=3), dict(groups=4, top_groups=5), dict(groups=0), dict(group_top=3),
                   dict(groups=8, top_groups=8, group_top=2), dict(groups=8, top_groups=1)):
            with pytest.raises(a2av.A2avError) as e:
                eng.route([x], [keys], [w], 2, **kw)
            assert e.value.code == a2av.ERR_INVALID_ARG, kw
        for kw in (dict(score="tanh"), dict(bias=torch.zeros(7, device="cuda")),
                   dict(counts=torch.zeros((1, 9), dtype=torch.int64, device="cuda"))):
            with pytest.raises(ValueError):
                eng.route([x], [keys], [w], 2, **kw)
        with pytest.raises(ValueError):
            eng.route([x.t()], [keys], [w], 2)  # not contiguous
        with pytest.raises(ValueError):
            eng.route([x.cpu()], [keys], [w], 2)
        with pytest.raises(ValueError):
            eng.route([x.double()], [keys], [w], 2)
        with pytest.raises(ValueError):
            eng.route([x], [keys.long()], [w], 2)
        with pytest.raises(ValueError):
            eng.route([x], [keys], [w], 3)
        with pytest.raises(ValueError):
            eng.route([x, x], [keys], [w], 2)
        wide = torch.randn((2, 1025), device="cuda")
        with pytest.raises(a2av.A2avError) as e:
            eng.route([wide], [keys[:2]], [w[:2]], 2)
        assert e.value.code == a2av.ERR_UNSUPPORTED
        cfg = a2av.A2avRoute(8, 2, a2av.F32, 0, 1, 1, 1, 1, 1.0)
        args = ([x.data_ptr()], [4], 0, [keys.data_ptr()], [w.data_ptr()], 0)
        assert a2av.a2av_route(eng.handle, cfg, *args) == a2av.OK
        for bad in (([0], [4], 0, [keys.data_ptr()], [w.data_ptr()], 0),
                    ([x.data_ptr() + 1], [4], 0, [keys.data_ptr()], [w.data_ptr()], 0),
                    ([x.data_ptr()], [-1], 0, [keys.data_ptr()], [w.data_ptr()], 0),
                    ([x.data_ptr()], [4], 2, [keys.data_ptr()], [w.data_ptr()], 0),
                    ([x.data_ptr()], [4], 0, [keys.data_ptr()], [w.data_ptr()], 4)):
            assert a2av.a2av_route(eng.handle, cfg, *bad) == a2av.ERR_INVALID_ARG
        torch.cuda.synchronize()
        assert eng.status() == a2av.OK
    assert a2av.load().a2av_route(None, ctypes.byref(cfg), None, None, None, None, None, None,
                                  None) == a2av.ERR_INVALID_ARG


@pytest.mark.parametrize("tokens", [(1, 0, 3), (8, 9, 0), (64, 1, 33), (65, 64, 130), (0, 700, 2047)])
@pytest.mark.parametrize("E,k", [(8, 2), (60, 3), (61, 3), (255, 7), (300, 8)])
def test_counts_of_uneven_ranks(tokens, E, k):
    """One block a rank or several; and ranks with fewer tokens than they were
    launched for, or none.  The counts are those of the keys, twice in a row into
    the same tensor."""
    W = len(tokens)
    gen = torch.Generator("cuda").manual_seed(sum(tokens) + E)
    counts = torch.full((W, E), 99, dtype=torch.int64, device="cuda")
    keys = [torch.empty(t, k, dtype=torch.int32, device="cuda") for t in tokens]
    weights = [torch.empty(t, k, device="cuda") for t in tokens]
    with a2av.A2av(W) as eng:
        for _ in range(2):
            logits = [torch.randn(t, E, device="cuda", generator=gen) for t in tokens]
            eng.route(logits, keys, weights, k, counts=counts)
            assert eng.status() == a2av.OK
            for r in range(W):
                assert torch.equal(logits[r].topk(k, dim=1).indices.int(), keys[r])
                assert torch.equal(torch.bincount(keys[r].view(-1).long(), minlength=E), counts[r])
