"""The workspaces that calls use when they are given none: calls that may be in
flight together (on two streams, from two threads, in a captured graph and
beside it) never share one, and a larger call takes none away."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()


class _Seen:
    """A module's functions; where the workspaces of the experts' gradients were."""

    def __init__(self, module):
        self._module, self.at = module, []

    def __getattr__(self, name):
        f = getattr(self._module, name)

        def seen(*args):
            result = f(*args)
            if name == "expert_matmul_backward" and result is not None:
                self.at.append(args[14].data_ptr())
            return result
        return seen


class _Product:
    """The gradients of a gated product: groups that are no multiples of 64 rows,
    so that dz and the packed remainders are both in the workspace."""

    def __init__(self, seed, rows=200, W=2, K=2, D=256, N=128):
        gen = torch.Generator("cuda").manual_seed(seed)
        new = lambda *shape: torch.randn(shape, device="cuda", generator=gen).bfloat16()
        self.counts = torch.randint(rows // 2, rows, (W, W * K), generator=gen, device="cuda")
        held = self.counts.view(W, W, K).sum((0, 2)).tolist()
        self.x = [new(m, D) for m in held]
        self.w = [new(K, 2 * N, D) for _ in range(W)]
        self.dy, self.pre = [new(m, N) for m in held], [new(m, 2 * N) for m in held]
        self.out = [[torch.empty_like(t) for t in ts] for ts in (self.x, self.w)]
        self.out.append([torch.empty(K, 2 * N, device="cuda").bfloat16() for _ in range(W)])
        self.shape = a2av.A2avExpert(K, D, N, a2av.BF16, 3, 1)
        self.need = a2av.a2av_expert_matmul_workspace_bytes(W, self.shape, sum(held))

    def call(self, eng, **options):
        eng.expert_matmul_backward(self.x, self.counts, self.w, self.dy, *self.out, pre=self.pre,
                                   activation="silu", gated=True, **options)

    def results(self):
        return [t.clone() for ts in self.out for t in ts]

    def expected(self, eng):
        """By itself, in a workspace of its own."""
        torch.cuda.synchronize()
        self.call(eng, workspace=torch.empty(self.need, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        expected = self.results()
        for ts in self.out:
            for t in ts:
                t.zero_()
        torch.cuda.synchronize()
        return expected


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def _where(eng, product, **options):
    """The workspace of a call: the first on a stream makes it, the second has it."""
    eng._marshal = seen = _Seen(a2av._marshal)
    product.call(eng, **options)
    product.call(eng, **options)
    torch.cuda.synchronize()
    return seen.at[-1]


def test_each_stream_and_each_thread_has_its_own():
    product = _Product(0)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with a2av.A2av(2) as eng:
        here = _where(eng, product)
        there = _where(eng, product, stream=side)
        with torch.cuda.stream(other):
            third = _where(eng, product)
        by_address = _where(eng, product, stream=other.cuda_stream)
        found = []
        thread = threading.Thread(target=lambda: found.append(_where(eng, product)))
        thread.start()
        thread.join()
        assert len({here, there, third, *found}) == 4
        assert by_address == third and _where(eng, product) == here
        assert eng.status() == a2av.OK


def test_two_streams_at_a_time():
    """Calls on two streams, the second's growing meanwhile: as each by itself."""
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sizes = (150, 400, 1500)
    products = [[_Product(10 * i + j, rows) for i, rows in enumerate(sizes)] for j in range(2)]
    with a2av.A2av(2) as eng:
        expected = [[p.expected(eng) for p in ps] for ps in products]
        for _ in range(3):
            for step in range(len(sizes)):
                for repeat in range(4):
                    for s, ps in zip(streams, products):
                        ps[step].call(eng, stream=s)
        torch.cuda.synchronize()
        assert eng.status() == a2av.OK
        for ps, es in zip(products, expected):
            for p, e in zip(ps, es):
                assert _same(p.results(), e)


def test_two_threads_on_one_stream():
    products = [_Product(20 + j, 300) for j in range(2)]
    with a2av.A2av(2) as eng:
        expected = [p.expected(eng) for p in products]
        start = threading.Barrier(2)

        def work(p):
            start.wait()
            for _ in range(50):
                p.call(eng)

        threads = [threading.Thread(target=work, args=(p,)) for p in products]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert eng.status() == a2av.OK
        for p, e in zip(products, expected):
            assert _same(p.results(), e)


@pytest.mark.parametrize("given", [False, True])
def test_a_captured_call_keeps_its_workspace(given):
    """Captured, then a larger call and allocations in between: the replay writes
    its own gradients and nothing of what was allocated since."""
    small, large = _Product(30, 150), _Product(31, 900)
    with a2av.A2av(2) as eng:
        expected, more = small.expected(eng), large.expected(eng)
        stream = torch.cuda.Stream()
        for _ in range(2):
            small.call(eng, stream=stream)  # (a kept workspace is there when the capture begins)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            small.call(eng, **(dict(stream=stream) if given else {}))
        large.call(eng, stream=stream)
        with torch.cuda.stream(stream):
            since = [torch.full((small.need,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        for ts in small.out:
            for t in ts:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            graph.replay()
            large.call(eng, stream=stream)  # (beside the replay, on the stream of the capture)
        torch.cuda.synchronize()
        assert eng.status() == a2av.OK
        assert _same(small.results(), expected) and _same(large.results(), more)
        assert all((t == 7).all() for t in since)


def test_given_workspaces_are_checked():
    """What is no contiguous memory of the device is refused, by the method as by
    the compiled checks; of another type, its bytes count."""
    product = _Product(40)
    need = product.need
    byte = lambda n, device="cuda": torch.zeros(n, dtype=torch.uint8, device=device)
    with a2av.A2av(2) as eng:
        expected = product.expected(eng)
        for module in (a2av._marshal, a2av._PlainMarshal):
            eng._marshal = module
            for bad in (byte(need, "cpu"), byte(need, "cpu").pin_memory(), byte(1).expand(need),
                        byte(2 * need)[::2], byte(need).cpu().numpy(), need):
                with pytest.raises(ValueError):
                    product.call(eng, workspace=bad)
            for small in (byte(need - 1), byte(0), torch.zeros((need - 1) // 4, device="cuda")):
                with pytest.raises(a2av.A2avError) as e:
                    product.call(eng, workspace=small)
                assert e.value.code == a2av.ERR_INVALID_ARG
            with pytest.raises(a2av.A2avError):
                product.call(eng, workspace=byte(need + 1)[1:])  # (not on 256 bytes)
            torch.cuda.synchronize()
            assert not any(t.any() for ts in product.out for t in ts)
            for good in (byte(need), torch.zeros((need + 3) // 4, dtype=torch.int32, device="cuda")):
                product.call(eng, workspace=good)
                assert _same(product.results(), expected)
                for ts in product.out:
                    for t in ts:
                        t.zero_()
        assert eng.status() == a2av.OK


class _Dispatch:
    """A dispatch of several kernels and its return path, rows of 8 bytes to 2 KiB."""

    def __init__(self, seed, tokens, width, W=4, K=4):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.W, self.K, self.width, m = W, K, width, 2 * tokens
        self.rows = [torch.randint(0, 256, (tokens, width), generator=gen, device="cuda").byte() for _ in range(W)]
        self.src = [torch.arange(tokens, device="cuda").int().repeat_interleave(2) for _ in range(W)]
        self.keys = [torch.randint(0, W * K, (m,), generator=gen, device="cuda").int() for _ in range(W)]
        to = torch.stack([torch.bincount(k // K, minlength=W) for k in self.keys])
        self.out = [torch.zeros(n, width, dtype=torch.uint8, device="cuda") for n in to.sum(0).tolist()]
        self.pos = [torch.zeros(m, dtype=torch.int64, device="cuda") for _ in range(W)]
        self.offsets = torch.zeros(W, 2, W, dtype=torch.int64, device="cuda")
        self.splits = torch.zeros(W, W, dtype=torch.int64, device="cuda")
        self.items = [torch.zeros(m, width, dtype=torch.uint8, device="cuda") for _ in range(W)]

    def arguments(self):
        return ((self.rows, self.src, self.keys, self.K, self.out, self.offsets, self.pos, self.width,
                 self.splits),
                (self.out, self.splits, self.keys, self.pos, self.K, self.items, self.width))

    def call(self, eng, **options):
        there, back = self.arguments()
        eng.dispatch(*there, **options)
        eng.combine_items(*back, **options)

    def check(self):
        for r in range(self.W):
            assert torch.equal(self.items[r], self.rows[r].repeat_interleave(2, 0))


@pytest.mark.parametrize("width", [8, 512, 2048])
def test_dispatches_on_two_streams(width):
    """Growing dispatches and their return paths on two streams at a time; bound
    on one stream and called on both; and captured, with a larger one after."""
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ds = [[_Dispatch(10 * i + j, n, width) for i, n in enumerate((300, 3000, 9000))] for j in range(2)]
    torch.cuda.synchronize()
    with a2av.A2av(4) as eng:
        for _ in range(3):
            for step in range(3):
                for s, d in zip(streams, ds):
                    d[step].call(eng, stream=s)
        torch.cuda.synchronize()
        assert eng.status() == a2av.OK
        for d in ds[0] + ds[1]:
            d.check()
        # bound on the first stream; the second's calls go with the second's workspaces
        bound = []
        for d in (ds[0][1], ds[1][1]):
            there, back = d.arguments()
            bound.append((eng.bind_dispatch(*there, stream=streams[0]),
                          eng.bind_combine_items(*back, stream=streams[0])))
            for t in d.items:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for s, calls in zip(streams, bound):
                for call in calls:
                    call(s)
        torch.cuda.synchronize()
        assert eng.status() == a2av.OK
        ds[0][1].check()
        ds[1][1].check()
        # captured, then a larger one on the same stream and allocations in between
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            ds[0][0].call(eng, stream=streams[0])
        larger = _Dispatch(77, 20000, width)
        for t in ds[0][0].items + larger.items:
            t.zero_()
        torch.cuda.synchronize()
        larger.call(eng, stream=streams[0])
        with torch.cuda.stream(streams[0]):
            since = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        for _ in range(2):
            graph.replay()
            larger.call(eng, stream=streams[0])
        torch.cuda.synchronize()
        assert eng.status() == a2av.OK
        ds[0][0].check()
        larger.check()
        assert all((t == 7).all() for t in since)


def test_given_workspaces_of_a_dispatch_are_checked():
    d = _Dispatch(5, 100, 64)
    need = a2av.a2av_dispatch_workspace_bytes(4, 4, 200)
    there, back = d.arguments()
    with a2av.A2av(4) as eng:
        for bad in (torch.zeros(need, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8, device="cuda").expand(need),
                    need):
            with pytest.raises(ValueError):
                eng.dispatch(*there, workspace=bad)
            with pytest.raises(ValueError):
                eng.combine_items(*back, workspace=bad)
        d.call(eng)
        assert eng.status() == a2av.OK
    d.check()
