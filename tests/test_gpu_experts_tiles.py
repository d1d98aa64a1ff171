"""The experts' products where every pair of CTAs takes several tiles: the ring of
stages, the tiles' descriptions and the two buffers of sums go round more than
once, with experts of many tiles of rows (more than one band of them), of one and
of none beside each other.  Against the definition in 64 bits; the bounds are those
of the arithmetic, as for small products."""
import math

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


def _act(name, z):
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z * 0.5 ** 0.5)
    return z / (1 + torch.exp(-z)) if name == "silu" else z.clamp_min(0) if name == "relu" else z


def _slope(name, z):
    if name == "gelu":
        return 0.5 * torch.erfc(-z * 0.5 ** 0.5) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return (z > 0).double() if name == "relu" else torch.ones_like(z)


def _one_long():
    """An expert of some 5000 rows from four ranks, none a multiple of 8: three bands."""
    return torch.tensor([[1501], [3], [2222], [1299]]).repeat(1, 4) * torch.tensor([1, 0, 0, 0])


def _mixed():
    """40 experts on two ranks: empty ones, of a few rows, of one tile, of several, of two bands."""
    gen = torch.Generator().manual_seed(2)
    sizes = torch.tensor([0, 0, 1, 9, 70, 130, 300, 700, 1400])
    return sizes[torch.randint(0, 9, (2, 40), generator=gen)]


def _full_and_empty():
    """Every other expert has no rows."""
    gen = torch.Generator().manual_seed(3)
    return torch.randint(1, 500, (2, 40), generator=gen) * (torch.arange(40) % 2)


def _many_groups():
    """256 experts on eight ranks: four groups to an entry of a block's table, which walks them."""
    gen = torch.Generator().manual_seed(4)
    return torch.randint(0, 24, (8, 256), generator=gen) * (torch.rand((8, 256), generator=gen) < 0.8)


COUNTS = {"one long": _one_long, "mixed": _mixed, "full and empty": _full_and_empty, "many groups": _many_groups}


class _Case:
    def __init__(self, kind, D, N, dtype, gated, seed=0):
        self.counts = COUNTS[kind]()
        self.W, E = self.counts.shape
        self.K, self.D, self.N, self.Z, self.dtype, self.gated = E // self.W, D, N, 2 * N if gated else N, dtype, gated
        gen = torch.Generator("cuda").manual_seed(seed)
        dt = moe.DTYPES[dtype]
        new = lambda *shape, std=1.0: (torch.randn(shape, device="cuda", generator=gen) * std).to(dt)
        held = self.counts.view(self.W, self.W, self.K).sum((0, 2)).tolist()
        self.x, self.w = [new(m, D) for m in held], [new(self.K, self.Z, D, std=D ** -0.5) for _ in held]
        self.b, self.res = [new(self.K, self.Z, std=0.3) for _ in held], [new(m, N) for m in held]
        self.dy, self.pre = [new(m, N) for m in held], [new(m, self.Z) for m in held]
        self.d_counts = self.counts.cuda()

    def row_tiles(self):
        """Tiles of rows of each expert: 32 granules of up to eight rows of one group."""
        return ((((self.counts + 7) // 8).sum(0) + 31) // 32)

    def experts(self):
        """(peer, expert, its rows in the peer's buffers)."""
        for p in range(self.W):
            groups = self.counts[:, p * self.K:(p + 1) * self.K].reshape(-1)
            owner = torch.arange(self.K).repeat(self.W).repeat_interleave(groups)
            for e in range(self.K):
                yield p, e, (owner == e).nonzero().view(-1).cuda()


def _pairs():
    return torch.cuda.get_device_properties(0).multi_processor_count // 2


def _close(got, ref, bound, dtype, what):
    limit = moe.UNIT[dtype] * (ref.abs() + bound) * 1.01 + moe.TINY[dtype] + bound
    off = (got.double() - ref).abs() > limit
    assert not bool(off.any()), f"{what}: {int(off.sum())} of {off.numel()} differ, first at {off.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name,gated", [("silu", True), ("gelu", False), ("none", False), ("relu", True)])
@pytest.mark.parametrize("kind,D,N", [("one long", 264, 2088), ("mixed", 200, 1032), ("full and empty", 520, 1288),
                                      ("many groups", 136, 264)])
def test_forward(kind, D, N, name, gated, dtype):
    c = _Case(kind, D, N, dtype, gated)
    tiles = int(c.row_tiles().sum()) * -(-N // (128 if gated else 256))
    assert tiles > 2 * _pairs()
    if kind in ("one long", "mixed"):
        assert c.row_tiles().max() > 8  # (more than a band)
    if kind == "mixed":
        assert {0, 1} <= set(c.row_tiles().tolist())
    full = name != "none"
    out = [torch.full_like(t, 7.0) for t in c.res]
    pre = [torch.full_like(t, 7.0) for t in c.pre]
    with a2av.A2av(c.W) as eng:
        eng.expert_matmul(c.x, c.d_counts, c.w, out, activation=name, gated=gated, bias=c.b if full else None,
                          residual=c.res if full else None, pre=pre)
        assert eng.status() == a2av.OK
    for p, e, at in c.experts():
        x, w, b = c.x[p][at].double(), c.w[p][e].double(), c.b[p][e].double() if full else 0.0
        z, size = x @ w.T + b, x.abs() @ w.abs().T + (b.abs() if full else 0.0)
        dz = (D + 8) * 2.0 ** -24 * size
        if gated:
            g, u = z[:, :N], z[:, N:]
            y = _act(name, g) * u
            bound = 1.13 * dz[:, :N] * (u.abs() + dz[:, N:]) + _act(name, g).abs() * dz[:, N:]
        else:
            y, bound = _act(name, z), 1.13 * dz
        bound = bound + 2.0 ** -16 * y.abs()  # (the activations' own error)
        if full:
            y = y + c.res[p][at].double()
        _close(out[p][at], y, bound + 2.0 ** -23 * y.abs(), dtype, f"peer {p} expert {e}")
        _close(pre[p][at], z, dz, dtype, f"pre of peer {p} expert {e}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name,gated", [("silu", True), ("gelu", False), ("none", False)])
@pytest.mark.parametrize("kind,D,N", [("one long", 2056, 1032), ("mixed", 1288, 520), ("full and empty", 1288, 264),
                                      ("many groups", 264, 136)])
def test_backward(kind, D, N, name, gated, dtype):
    c = _Case(kind, D, N, dtype, gated, seed=1)
    nd = -(-D // 256)
    assert int(c.row_tiles().sum()) * nd > 2 * _pairs()  # of the rows' gradient
    assert c.W * c.K * -(-c.Z // 256) * nd > 2 * _pairs()  # of the weights'
    plain = name == "none" and not gated
    d_x, d_w = [torch.full_like(t, 7.0) for t in c.x], [torch.full_like(t, 7.0) for t in c.w]
    d_b = [torch.full_like(t, 7.0) for t in c.b]
    with a2av.A2av(c.W) as eng:
        eng.expert_matmul_backward(c.x, c.d_counts, c.w, c.dy, d_x, d_w, d_b, pre=None if plain else c.pre,
                                   activation=name, gated=gated)
        assert eng.status() == a2av.OK
    for p, e, at in c.experts():
        x, w, dy, z = c.x[p][at].double(), c.w[p][e].double(), c.dy[p][at].double(), c.pre[p][at].double()
        if gated:
            dz = torch.cat([dy * z[:, N:] * _slope(name, z[:, :N]), dy * _act(name, z[:, :N])], 1)
            # (a slope is a sum of two terms: its error goes by them)
            size = torch.cat([(dy * z[:, N:]).abs() * (1 + z[:, :N].abs()), dz[:, N:].abs()], 1)
        else:
            dz = dy * _slope(name, z)
            size = dy.abs() if plain else dy.abs() * (1 + z.abs())
        # dz is rounded to the type (not where it is dy itself), the sums are of 32 bits
        off = 0.0 if plain else moe.UNIT[dtype] * 1.01
        dz_off = off * dz.abs() + (0.0 if plain else 2.0 ** -16 * size + moe.TINY[dtype])
        m = at.numel()
        _close(d_x[p][at], dz @ w, dz_off @ w.abs() + (c.Z + 8) * 2.0 ** -24 * (dz.abs() @ w.abs()), dtype,
               f"d_rows {p} {e}")
        _close(d_w[p][e], dz.T @ x, dz_off.T @ x.abs() + (m + 8) * 2.0 ** -24 * (dz.abs().T @ x.abs()), dtype,
               f"d_weights {p} {e}")
        _close(d_b[p][e], dz.sum(0), dz_off.sum(0) + (m + 8) * 2.0 ** -24 * dz.abs().sum(0), dtype, f"d_bias {p} {e}")


def test_repeats_itself_and_in_a_graph():
    """The same bits each time, in a captured call too, forward and backward."""
    c = _Case("mixed", 264, 520, "bf16", True, seed=2)
    new = lambda like: [torch.empty_like(t) for t in like]
    outs = [new(c.res), new(c.pre), new(c.x), new(c.w), new(c.b)]
    with a2av.A2av(c.W) as eng:
        def step(stream=None):
            eng.expert_matmul(c.x, c.d_counts, c.w, outs[0], activation="silu", gated=True, bias=c.b,
                              residual=c.res, pre=outs[1], stream=stream)
            eng.expert_matmul_backward(c.x, c.d_counts, c.w, c.dy, *outs[2:], pre=outs[1], activation="silu",
                                       gated=True, stream=stream)
        step()
        torch.cuda.synchronize()
        first = [t.clone() for ts in outs for t in ts]
        graph = torch.cuda.CUDAGraph()
        stream = torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            step(stream)
        for run in (step, graph.replay, graph.replay):
            for ts in outs:
                for t in ts:
                    t.fill_(7.0)
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            assert eng.status() == a2av.OK
            assert all(torch.equal(a, b) for a, b in zip(first, [t for ts in outs for t in ts]))
