"""The weighted combine on the GPU: outputs and gradients against the
definition in 64 bits, its layout against the dispatch's, and what it refuses."""
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


def _case(T, K, k, H, dtype, seed, offset=0):
    """Random items in the dispatch's layout; buffers start `offset` elements past 16 bytes."""
    W, rng = len(T), np.random.default_rng(seed)
    dt = moe.DTYPES[dtype]
    E = W * K
    keys = [np.stack([rng.permutation(E)[:k] for _ in range(n)]).reshape(n, k) if n else np.zeros((0, k), int)
            for n in T]
    S = np.zeros((W, W), np.int64)
    pos = []
    for r, x in enumerate(keys):
        flat = x.reshape(-1)
        order = np.argsort(flat, kind="stable")
        q = np.empty(flat.size, np.int64)
        q[order] = np.arange(flat.size)
        pos.append(q)
        S[r] = np.bincount(flat // K, minlength=W)

    def place(values):
        buf = torch.empty(values.size + offset, dtype=dt, device="cuda")
        view = buf[offset:].view(values.shape)
        view.copy_(torch.from_numpy(values))
        return view

    c = {"W": W, "K": K, "k": k, "H": H, "S": S, "keys": keys, "pos": pos, "T": T, "dtype": dtype,
         "peers": [place(rng.standard_normal((int(S[:, p].sum()), H))) for p in range(W)],
         "weights": [torch.from_numpy(rng.random((n, k)).astype(np.float32)).cuda() for n in T],
         "residual": [place(rng.standard_normal((n, H))) for n in T],
         "dy": [place(rng.standard_normal((n, H))) for n in T], "place": place}
    c["d_S"] = torch.from_numpy(S).cuda()
    c["d_keys"] = [torch.from_numpy(x.astype(np.int32)).cuda() for x in keys]
    c["d_pos"] = [torch.from_numpy(x).cuda() for x in pos]
    return c


def _rows_of(c, r):
    """(peer, row in the peer's buffer) of each of rank r's items."""
    S, K = c["S"], c["K"]
    peer = c["keys"][r].reshape(-1) // K
    return peer, np.array([S[:r, p].sum() + q - S[r, :p].sum() for p, q in zip(peer, c["pos"][r])],
                          dtype=np.int64)


SHAPES = [([1], 1, 1, 8), ([1], 4, 2, 7168), ([5, 0, 3], 2, 3, 64), ([33, 1], 8, 2, 1000),
          ([7, 7], 3, 6, 65), ([1, 0], 5, 1, 1), ([50, 49, 3, 8], 16, 2, 513), ([2] * 8, 8, 4, 2056),
          ([3], 32, 32, 40), ([300], 2, 1, 24), ([600, 500], 8, 2, 512), ([200] * 8, 8, 3, 1544)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, offset, dtype):
    c = _case(*shape, dtype, 1, offset)
    W, K, k, H = c["W"], c["K"], c["k"], c["H"]
    x64 = [moe.f64(x) for x in c["peers"]]
    for weighted in (True, False):
        for residual in (True, False):
            out = [c["place"](np.full((n, H), 7.0)) for n in c["T"]]
            with a2av.A2av(W) as eng:
                eng.combine_weighted(c["peers"], c["d_S"], c["d_keys"], c["d_pos"], K,
                                     c["weights"] if weighted else None, out,
                                     residual=c["residual"] if residual else None)
                assert eng.status() == a2av.OK
            for r, n in enumerate(c["T"]):
                peer, row = _rows_of(c, r)
                w = moe.f64(c["weights"][r]).reshape(-1) if weighted else np.ones(n * k)
                terms = np.array([w[i] * x64[peer[i]][row[i]] for i in range(n * k)]).reshape(n, k, H)
                ref, mag = terms.sum(1), np.abs(terms).sum(1)
                if residual:
                    ref, mag = ref + moe.f64(c["residual"][r]), mag + np.abs(moe.f64(c["residual"][r]))
                moe.close(out[r], ref, (k + 2) * 2.0 ** -24 * mag, dtype, f"rank {r}")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, offset, dtype):
    c = _case(*shape, dtype, 2, offset)
    W, K, k, H = c["W"], c["K"], c["k"], c["H"]
    x64 = [moe.f64(x) for x in c["peers"]]
    for rows, weights in ((True, True), (True, False), (False, True)):
        d_peers = [c["place"](np.full(tuple(x.shape), 7.0)) for x in c["peers"]] if rows else None
        d_w = [torch.full((n, k), 7.0, device="cuda") for n in c["T"]] if weights else None
        with a2av.A2av(W) as eng:
            eng.combine_weighted_backward(c["peers"] if weights else None, c["d_S"], c["d_keys"],
                                          c["d_pos"], K, c["weights"], c["dy"], d_peers, d_w)
            assert eng.status() == a2av.OK
        seen = [np.zeros(x.shape[0], int) for x in x64]
        for r, n in enumerate(c["T"]):
            peer, row = _rows_of(c, r)
            dy, w = moe.f64(c["dy"][r]), moe.f64(c["weights"][r]).reshape(-1)
            for i in range(n * k):
                p, q = peer[i], row[i]
                seen[p][q] += 1
                if rows:
                    ref = w[i] * dy[i // k]
                    moe.close(d_peers[p][q], ref, 2.0 ** -24 * np.abs(ref), dtype, "d_peers")
            if weights and n:
                t = np.repeat(dy, k, axis=0)
                x = np.array([x64[p][q] for p, q in zip(peer, row)])
                ref, mag = (t * x).sum(1), np.abs(t * x).sum(1)
                moe.close(d_w[r].reshape(-1), ref, (H + 4) * 2.0 ** -24 * mag, "f32", "d_weights")
        assert all((s == 1).all() for s in seen)


def test_gradient_against_differences():
    """<dy, out(x + h v) - out(x - h v)> / 2h against <d_peers, v> and the weights' likewise."""
    c = _case([6, 4], 3, 2, 48, "f32", 4)
    W, K, k = c["W"], c["K"], c["k"]

    def out(peers, weights):
        y = [torch.empty_like(t) for t in c["dy"]]
        with a2av.A2av(W) as eng:
            eng.combine_weighted(peers, c["d_S"], c["d_keys"], c["d_pos"], K, weights, y)
            assert eng.status() == a2av.OK
        return sum((a.double() * b.double()).sum().item() for a, b in zip(y, c["dy"]))

    d_peers = [torch.empty_like(x) for x in c["peers"]]
    d_w = [torch.empty_like(x) for x in c["weights"]]
    with a2av.A2av(W) as eng:
        eng.combine_weighted_backward(c["peers"], c["d_S"], c["d_keys"], c["d_pos"], K, c["weights"],
                                      c["dy"], d_peers, d_w)
        assert eng.status() == a2av.OK
    for xs, ds, which in ((c["peers"], d_peers, 0), (c["weights"], d_w, 1)):
        v = [torch.randn_like(x) for x in xs]
        hi, lo = [x + 0.5 * a for x, a in zip(xs, v)], [x - 0.5 * a for x, a in zip(xs, v)]
        a, b = (out(hi, c["weights"]), out(lo, c["weights"])) if which == 0 else \
            (out(c["peers"], hi), out(c["peers"], lo))
        want = sum((d.double() * t.double()).sum().item() for d, t in zip(ds, v))
        size = sum((d.double() * t.double()).abs().sum().item() for d, t in zip(ds, v))
        assert abs((a - b) - want) <= 2.0 ** -18 * (size + abs(a) + abs(b))  # linear: no step error


def test_inverse_of_the_dispatch():
    """dispatch, then combine_weighted with weights that sum to 1: every token's own row again."""
    W, K, n, k, H = 4, 4, 900, 2, 72
    rng = np.random.default_rng(0)
    rows = [torch.randn((n, H), device="cuda") for _ in range(W)]
    x = [torch.randn((n, W * K), device="cuda") for _ in range(W)]
    keys = [torch.empty((n, k), dtype=torch.int32, device="cuda") for _ in range(W)]
    w = [torch.empty((n, k), device="cuda") for _ in range(W)]
    counts = torch.empty((W, W * K), dtype=torch.int64, device="cuda")
    src = [torch.arange(n, dtype=torch.int32, device="cuda").repeat_interleave(k) for _ in range(W)]
    pos = [torch.empty(n * k, dtype=torch.int64, device="cuda") for _ in range(W)]
    so = torch.empty((W, 2, W), dtype=torch.int64, device="cuda")
    S = torch.empty((W, W), dtype=torch.int64, device="cuda")
    with a2av.A2av(W) as eng:
        eng.route(x, keys, w, k, counts=counts)
        held = counts.view(W, W, K).sum((0, 2)).tolist()
        out = [torch.empty((m, H), device="cuda") for m in held]
        eng.dispatch([r.view(-1).view(torch.uint8) for r in rows], src, keys, K, [o.view(torch.uint8) for o in out],
                     so, pos, H * 4, in_splits=S)
        y = [torch.empty((n, H), device="cuda") for _ in range(W)]
        eng.combine_weighted(out, S, keys, pos, K, w, y)
        assert eng.status() == a2av.OK
    assert torch.equal(S, counts.view(W, W, K).sum(2))
    for a, b in zip(y, rows):
        assert (a - b).abs().max() <= 2.0 ** -21 * b.abs().max()


def test_residual_in_place_and_other_stream():
    c = _case([20, 9], 4, 2, 128, "bf16", 6)
    ref = [torch.empty_like(x) for x in c["residual"]]
    s = torch.cuda.Stream()
    with a2av.A2av(2) as eng:
        args = (c["peers"], c["d_S"], c["d_keys"], c["d_pos"], c["K"], c["weights"])
        eng.combine_weighted(*args, ref, residual=c["residual"])
        torch.cuda.synchronize()
        s.wait_stream(torch.cuda.current_stream())
        call = eng.bind_combine_weighted(*args, c["residual"], residual=c["residual"], stream=s)
        call()
        assert eng.status(s) == a2av.OK
    assert all(torch.equal(a, b) for a, b in zip(ref, c["residual"]))


def test_invalid_items_and_splits():
    c = _case([4, 3], 2, 2, 32, "f32", 7)
    out = [torch.full((n, 32), 7.0, device="cuda") for n in c["T"]]
    with a2av.A2av(2) as eng:
        args = lambda S, keys, pos: (c["peers"], S, keys, pos, c["K"], c["weights"], out)
        keys = [c["d_keys"][0].clone(), c["d_keys"][1]]
        keys[0][1, 1] = 4
        eng.combine_weighted(*args(c["d_S"], keys, c["d_pos"]))
        assert eng.status() == a2av.ERR_BAD_INDEX
        assert (out[0][1] == 7).all() and not (out[0][0] == 7).any() and not (out[1] == 7).any()
        pos = [c["d_pos"][0], c["d_pos"][1].clone()]
        pos[1][0] = -1
        out[1].fill_(7)
        eng.combine_weighted(*args(c["d_S"], c["d_keys"], pos))
        assert eng.status() == a2av.ERR_BAD_INDEX
        assert (out[1][0] == 7).all() and not (out[1][1:] == 7).any()
        for r, p, by in ((0, 0, 1), (1, 1, -100)):
            S = c["d_S"].clone()
            S[r, p] += by
            for o in out:
                o.fill_(7)
            eng.combine_weighted(*args(S, c["d_keys"], c["d_pos"]))
            assert eng.status() == a2av.ERR_BAD_SPLITS
            assert all((o == 7).all() for o in out)


def test_refusals():
    c = _case([4], 2, 2, 32, "f32", 8)
    out = [torch.empty((4, 32), device="cuda")]
    with a2av.A2av(1) as eng:
        good = dict(peers=c["peers"], in_splits=c["d_S"], keys=c["d_keys"], sorted_pos=c["d_pos"],
                    keys_per_peer=2, weights=c["weights"], outputs=out)
        for change in (dict(peers=[c["peers"][0].half()]), dict(peers=[c["peers"][0][:, :31]]),
                       dict(in_splits=c["d_S"].int()), dict(keys=[c["d_keys"][0].long()]),
                       dict(sorted_pos=[c["d_pos"][0][:-1]]), dict(weights=[c["weights"][0][:, :1]]),
                       dict(outputs=[out[0].double()]), dict(outputs=[out[0].cpu()]),
                       dict(residual=[out[0][:3]]), dict(peers=c["peers"] * 2)):
            with pytest.raises(ValueError):
                eng.combine_weighted(**{**good, **change})
        for K, code in ((0, a2av.ERR_INVALID_ARG), (1025, a2av.ERR_UNSUPPORTED)):
            with pytest.raises(a2av.A2avError) as e:
                eng.combine_weighted(**{**good, "keys_per_peer": K})
            assert e.value.code == code
        with pytest.raises(ValueError):
            eng.combine_weighted_backward(c["peers"], c["d_S"], c["d_keys"], c["d_pos"], 2,
                                          c["weights"], c["dy"])
        with pytest.raises(ValueError):
            eng.combine_weighted_backward(None, c["d_S"], c["d_keys"], c["d_pos"], 2, c["weights"],
                                          c["dy"], None, [torch.empty((4, 2), device="cuda")])
        assert eng.status() == a2av.OK
    assert a2av.a2av_combine_weighted(None, 1, 1, 1, 0, [], [], 0, [], [], None, [], None, []) \
        == a2av.ERR_INVALID_ARG
