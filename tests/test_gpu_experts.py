"""The experts' products on the GPU: results and gradients against the
definition in 64 bits, with error bounds from the arithmetic, and what they
refuse."""
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


def _counts(rng, W, K, rows, kind):
    """Items of each (rank, expert): `rows` a group on average."""
    E = W * K
    if kind == "empty":
        return np.zeros((W, E), np.int64)
    if kind == "one":
        c = np.zeros((W, E), np.int64)
        c[rng.integers(W), rng.integers(E)] = rows
        return c
    c = rng.integers(0, 2 * rows + 1, (W, E))
    if kind == "sparse":
        c = c * (rng.random((W, E)) < 0.4)
    return c.astype(np.int64)


def _case(W, K, D, N, rows, dtype, gated, kind="random", seed=0, offset=0, slack=0, pre=False):
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

    c = {"W": W, "K": K, "D": D, "N": N, "Z": Z, "counts": counts, "held": held, "dtype": dtype,
         "gated": gated, "place": place, "d_counts": torch.from_numpy(counts).cuda(),
         "x": [place(rng.standard_normal((m, D))) for m in held],
         "w": [place(rng.standard_normal((K, Z, D)) * D ** -0.5) for _ in range(W)],
         "b": [place(rng.standard_normal((K, Z)) * 0.3) for _ in range(W)],
         "res": [place(rng.standard_normal((m, N))) for m in held],
         "dy": [place(rng.standard_normal((m, N))) for m in held],
         "owner": [moe.row_experts(counts, p, K) for p in range(W)]}
    if pre:
        c["pre"] = [place(rng.standard_normal((m, Z))) for m in held]
    return c


def _forward(c, name, bias, residual, pre=True, stream=None, x=None):
    out = [c["place"](np.full((m, c["N"]), 7.0)) for m in c["held"]]
    saved = [c["place"](np.full((m, c["Z"]), 7.0)) for m in c["held"]] if pre else None
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    with a2av.A2av(c["W"]) as eng:
        eng.expert_matmul(x or c["x"], c["d_counts"], c["w"], out, activation=name, gated=c["gated"],
                          bias=c["b"] if bias else None, residual=c["res"] if residual else None,
                          pre=saved, stream=stream)
        assert eng.status(stream) == a2av.OK
    return out, saved


def _check_forward(c, name, bias, residual, out, saved):
    for p in range(c["W"]):
        n = c["owner"][p].size
        y, z, bound, dz = moe.expert_forward(
            moe.f64(c["x"][p])[:n], c["owner"][p], moe.f64(c["w"][p]), moe.f64(c["b"][p]) if bias else None,
            moe.f64(c["res"][p])[:n] if residual else None, name, c["gated"])
        bound = bound + 2.0 ** -23 * np.abs(y)
        moe.close(out[p][:n], y, bound, c["dtype"], f"peer {p}")
        assert (out[p][n:] == 7).all(), "rows past the groups written"
        if saved is not None:
            moe.close(saved[p][:n], z, dz, c["dtype"], f"pre of peer {p}")
            assert (saved[p][n:] == 7).all()


# (W, K, D, N, rows of a group on average)
SHAPES = [(1, 1, 64, 128, 1), (1, 1, 64, 128, 300), (2, 3, 128, 72, 20), (1, 4, 200, 264, 70),
          (4, 2, 72, 40, 9), (1, 1, 8, 8, 5), (1, 2, 1000, 136, 129), (2, 2, 320, 512, 40),
          (1, 1, 33, 17, 50), (2, 2, 65, 64, 30), (1, 3, 64, 63, 10), (8, 8, 64, 64, 3),
          (1, 1, 2048, 256, 2)]
EPILOGUES = [("none", False, False, False), ("silu", True, False, False), ("gelu", False, True, True),
             ("relu", False, True, False), ("silu", False, False, True), ("gelu", True, True, True),
             ("none", True, True, False), ("none", False, False, True)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("epilogue", EPILOGUES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, epilogue, dtype):
    name, gated, bias, residual = epilogue
    c = _case(*shape, dtype, gated, seed=1, slack=3)
    _check_forward(c, name, bias, residual, *_forward(c, name, bias, residual))


@pytest.mark.parametrize("kind", ["empty", "one", "sparse"])
@pytest.mark.parametrize("gated", [False, True])
def test_forward_uneven_groups(kind, gated):
    c = _case(3, 4, 96, 80, 150, "bf16", gated, kind, seed=2, slack=1)
    _check_forward(c, "silu", True, False, *_forward(c, "silu", True, False))


@pytest.mark.parametrize("offset", [1, 4])
def test_forward_unaligned_buffers(offset):
    c = _case(2, 2, 128, 64, 33, "f16", True, seed=3, offset=offset)
    _check_forward(c, "silu", True, True, *_forward(c, "silu", True, True))


def test_many_groups():
    """More groups than a block's table has entries: 32 ranks, 32 experts each."""
    rng = np.random.default_rng(0)
    c = _case(32, 32, 32, 16, 1, "bf16", False, "sparse", seed=4)
    _check_forward(c, "none", False, False, *_forward(c, "none", False, False, pre=False), )


def test_rows_of_nan_stay_within_their_results():
    """NaN and infinities in one group, and in the slack past the groups, reach no other row."""
    c = _case(1, 3, 128, 64, 40, "bf16", False, "random", seed=5, slack=2)
    n = c["owner"][0].size
    clean, _ = _forward(c, "none", True, False)
    x = c["x"][0].clone()
    x[n:] = float("nan")
    bad = np.nonzero(c["owner"][0] == 1)[0]
    x[torch.from_numpy(bad).cuda()] = float("inf")
    out, _ = _forward(c, "none", True, False, x=[x])
    other = torch.from_numpy(np.nonzero(c["owner"][0] != 1)[0]).cuda()
    assert torch.equal(out[0][other], clean[0][other])
    # and the weights' gradients: the other experts' stay finite and equal
    grads = []
    for rows in (c["x"][0], x):
        d_w = [torch.empty_like(c["w"][0])]
        with a2av.A2av(1) as eng:
            eng.expert_matmul_backward([rows], c["d_counts"], c["w"], c["dy"], d_weights=d_w)
            assert eng.status() == a2av.OK
        grads.append(d_w[0])
    for e in (0, 2):
        assert torch.equal(grads[0][e], grads[1][e]) and torch.isfinite(grads[1][e]).all()


def _check_backward(c, name, bias, rows=True, weights=True):
    new = lambda like: [c["place"](np.full(tuple(t.shape), 7.0)) for t in like]
    d_x, d_w, d_b = new(c["x"]) if rows else None, new(c["w"]) if weights else None, new(c["b"]) if bias else None
    pre = c["pre"] if name != "none" or c["gated"] else None
    with a2av.A2av(c["W"]) as eng:
        eng.expert_matmul_backward(c["x"], c["d_counts"], c["w"], c["dy"], d_rows=d_x, d_weights=d_w,
                                   d_bias=d_b, pre=pre, activation=name, gated=c["gated"])
        assert eng.status() == a2av.OK
    u = moe.UNIT[c["dtype"]]
    for p in range(c["W"]):
        n, owner = c["owner"][p].size, c["owner"][p]
        dz = moe.expert_dz(moe.f64(c["dy"][p])[:n], None if pre is None else moe.f64(pre[p])[:n], name, c["gated"])
        x, w = moe.f64(c["x"][p])[:n], moe.f64(c["w"][p])
        # dz is rounded to the type (not where it is dy itself), the sums are of 32 bits
        off = 0 if pre is None else u * 1.01 + 2.0 ** -17
        least = 0 if pre is None else moe.TINY[c["dtype"]] + 2.0 ** -21 * np.abs(dz).max(initial=0)
        mag = np.abs(dz)
        for e in range(c["K"]):
            at = owner == e
            if rows:
                size = mag[at] @ np.abs(w[e])
                bound = (off + (c["Z"] + 8) * 2.0 ** -24) * size + least * np.abs(w[e]).sum(0)
                moe.close(d_x[p][:n][torch.from_numpy(at).cuda()], dz[at] @ w[e], bound, c["dtype"], "d_rows")
            m = int(at.sum())
            if weights:
                size = mag[at].T @ np.abs(x[at])
                bound = (off + (m + 8) * 2.0 ** -24) * size + least * np.abs(x[at]).sum(0)
                moe.close(d_w[p][e], dz[at].T @ x[at], bound, c["dtype"], f"d_weights {p} {e}")
            if bias:
                bound = (off + (m + 8) * 2.0 ** -24) * mag[at].sum(0) + least * m
                moe.close(d_b[p][e], dz[at].sum(0), bound, c["dtype"], "d_bias")
        if rows:
            assert (d_x[p][n:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("epilogue", EPILOGUES[:7], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, epilogue, dtype):
    name, gated, bias, _ = epilogue
    _check_backward(_case(*shape, dtype, gated, seed=6, slack=2, pre=True), name, bias)


@pytest.mark.parametrize("kind", ["empty", "one", "sparse"])
def test_backward_uneven_groups(kind):
    """Experts without rows get gradients of 0."""
    _check_backward(_case(3, 4, 96, 80, 150, "bf16", True, kind, seed=7, pre=True), "silu", True)


def test_backward_parts_and_unaligned_buffers():
    c = _case(2, 2, 128, 64, 33, "bf16", False, seed=8, pre=True)
    _check_backward(c, "gelu", False, rows=True, weights=False)
    _check_backward(c, "gelu", False, rows=False, weights=True)
    _check_backward(_case(2, 2, 128, 64, 33, "bf16", False, seed=8, offset=1, pre=True), "gelu", True)


@pytest.mark.parametrize("name", ["relu", "gelu", "silu", "none"])
def test_dz_formula_against_differences(name):
    """The definition's dz against central differences of its y (64 bits)."""
    rng = np.random.default_rng(1)
    z, dy, h = rng.standard_normal((5, 12)), rng.standard_normal((5, 6)), 1e-6
    for gated in (False, True):
        d = dy if gated else np.concatenate([dy, dy], 1)
        f = (lambda z: moe.act(name, z[:, :6]) * z[:, 6:]) if gated else (lambda z: moe.act(name, z))
        got = moe.expert_dz(d, z, name, gated)
        for i in range(12):
            e = np.zeros(12)
            e[i] = h
            num = ((f(z + e) - f(z - e)) * d).sum(1) / (2 * h)
            assert np.abs(num - got[:, i]).max() < 1e-7


def test_forward_then_backward_against_differences():
    """<dy, y(x + v) - y(x - v)> against <d_rows, v> for a product without activation (linear)."""
    c = _case(2, 2, 256, 128, 40, "f16", False, seed=9)
    d_x = [torch.empty_like(x) for x in c["x"]]
    with a2av.A2av(2) as eng:
        eng.expert_matmul_backward(c["x"], c["d_counts"], c["w"], c["dy"], d_rows=d_x)
        assert eng.status() == a2av.OK
    v = [torch.randn_like(x) for x in c["x"]]
    hi, _ = _forward(c, "none", False, False, x=[a + b for a, b in zip(c["x"], v)])
    lo, _ = _forward(c, "none", False, False, x=[a - b for a, b in zip(c["x"], v)])
    a = sum(((p.double() - q.double()) * d.double()).sum().item() for p, q, d in zip(hi, lo, c["dy"])) / 2
    b = sum((d.double() * t.double()).sum().item() for d, t in zip(d_x, v))
    size = sum((d.double() * t.double()).square().sum().item() for d, t in zip(d_x, v)) ** 0.5
    size += sum((p.double() * d.double()).square().sum().item() for p, d in zip(hi + lo, c["dy"] * 2)) ** 0.5
    assert abs(a - b) <= 16 * 2.0 ** -11 * size  # roundings to 11 bits, as a random walk


def test_deterministic_and_other_stream():
    c = _case(2, 4, 512, 256, 100, "bf16", True, seed=10)
    first, _ = _forward(c, "silu", True, True)
    again, _ = _forward(c, "silu", True, True, pre=False, stream=torch.cuda.Stream())
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_bound_call_with_new_counts():
    """A bound call takes new counts and rows in the same buffers."""
    c = _case(1, 2, 64, 32, 30, "bf16", False, seed=11)
    out = [torch.empty((c["held"][0], 32), dtype=torch.bfloat16, device="cuda")]
    with a2av.A2av(1) as eng:
        call = eng.bind_expert_matmul(c["x"], c["d_counts"], c["w"], out)
        call()
        n = c["held"][0]
        for split in ([n, 0], [1, n - 1], [0, 1]):
            c["d_counts"].copy_(torch.tensor([split]))
            out[0].fill_(7)
            call()
            assert eng.status() == a2av.OK
            c["counts"] = np.array([split])
            c["owner"] = [moe.row_experts(c["counts"], 0, 2)]
            _check_forward(c, "none", False, False, out, None)


def test_residual_in_place():
    c = _case(1, 2, 64, 96, 60, "bf16", False, seed=12)
    ref, _ = _forward(c, "relu", True, True)
    with a2av.A2av(1) as eng:
        eng.expert_matmul(c["x"], c["d_counts"], c["w"], c["res"], activation="relu", bias=c["b"],
                          residual=c["res"])
        assert eng.status() == a2av.OK
    assert torch.equal(ref[0], c["res"][0])


def test_invalid_counts_write_nothing():
    c = _case(2, 2, 64, 32, 20, "bf16", False, seed=13)
    out = [torch.full((m, 32), 7.0, dtype=torch.bfloat16, device="cuda") for m in c["held"]]
    d_w = [torch.full_like(w, 7.0) for w in c["w"]]
    with a2av.A2av(2) as eng:
        for r, e, by in ((0, 0, 1), (1, 3, -1000), (0, 2, 1 << 40)):
            counts = c["d_counts"].clone()
            counts[r, e] += by
            eng.expert_matmul(c["x"], counts, c["w"], out)
            assert eng.status() == a2av.ERR_BAD_SPLITS
            eng.expert_matmul_backward(c["x"], counts, c["w"], c["dy"], d_rows=out if False else None,
                                       d_weights=d_w)
            assert eng.status() == a2av.ERR_BAD_SPLITS
            assert all((o == 7).all() for o in out + d_w)


def test_refusals():
    c = _case(1, 2, 64, 32, 10, "bf16", False, seed=14)
    out = [torch.empty((c["held"][0], 32), dtype=torch.bfloat16, device="cuda")]
    good = dict(rows=c["x"], counts=c["d_counts"], weights=c["w"], outputs=out)
    with a2av.A2av(1) as eng:
        for change in (dict(rows=[c["x"][0].float()]), dict(rows=[c["x"][0].half()]), dict(rows=[c["x"][0][:, :63]]),
                       dict(weights=[c["w"][0][:, :, :63]]), dict(weights=[c["w"][0].float()]),
                       dict(weights=[None]), dict(counts=c["d_counts"].int()),
                       dict(counts=torch.zeros((1, 3), dtype=torch.int64, device="cuda")),
                       dict(outputs=[out[0][:-1]]), dict(outputs=[out[0].t()]), dict(activation="tanh"),
                       dict(gated=True), dict(bias=[c["b"][0][:1]]), dict(residual=[out[0][:-1]]),
                       dict(pre=[out[0].float()])):
            with pytest.raises(ValueError):
                eng.expert_matmul(**{**good, **change})
        with pytest.raises(ValueError):
            eng.expert_matmul_backward(c["x"], c["d_counts"], c["w"], c["dy"], activation="silu",
                                       d_rows=[torch.empty_like(c["x"][0])])
        with pytest.raises(a2av.A2avError) as e:
            eng.expert_matmul_backward(c["x"], c["d_counts"], c["w"], c["dy"])
        assert e.value.code == a2av.ERR_INVALID_ARG
        shape = a2av.A2avExpert(2, 64, 32, a2av.F32, 0, 0)
        assert a2av.a2av_expert_matmul_workspace_bytes(1, shape, 10) == -1
        shape = a2av.A2avExpert(2, 64, 32, a2av.BF16, 3, 1)
        # dz, and the packed remainders of dz and x: at most every row, and 63 rows of zeros an expert
        assert a2av.a2av_expert_matmul_workspace_bytes(1, shape, 10) == 10 * 64 * 2 + (10 + 2 * 63) * (64 + 64) * 2
        assert a2av.a2av_expert_matmul_workspace_bytes(1, shape, -1) == -1
        assert a2av.a2av_expert_matmul_workspace_bytes(1, shape, 1 << 31) == -1
        n, ptr = c["held"], lambda ts: [t.data_ptr() for t in ts]
        call = lambda shape, **kw: a2av.a2av_expert_matmul(
            eng.handle, shape, kw.get("x", ptr(c["x"])), kw.get("n", n), kw.get("c", c["d_counts"].data_ptr()),
            ptr(c["w"]), None, None, ptr(out), None)
        ok = lambda **kw: a2av.A2avExpert(*[{**dict(K=2, D=64, N=32, t=a2av.BF16, a=0, g=0), **kw}[i] for i in "KDNtag"])
        assert call(ok()) == a2av.OK
        for bad in (call(ok(K=0)), call(ok(D=0)), call(ok(N=0)), call(ok(t=0)), call(ok(a=4)), call(ok(), x=[0]),
                    call(ok(), n=[-1]), call(ok(), c=0), call(ok(), x=[c["x"][0].data_ptr() + 1])):
            assert bad == a2av.ERR_INVALID_ARG
        assert call(ok(K=1025)) == a2av.ERR_UNSUPPORTED and call(ok(D=1 << 25)) == a2av.ERR_UNSUPPORTED
        assert eng.status() == a2av.OK
