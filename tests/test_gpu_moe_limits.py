"""The most tokens and rows that a call takes, 2^31 - 1, where a 32-bit count that
goes on by a grid's stride would wrap: every value of every output, exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")

MOST = 2 ** 31 - 1
PART = 1 << 27


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("less than 120 GB free")
    yield
    torch.cuda.empty_cache()


def _pattern(first, n):
    """-1, 0 or 2 by the position, of no period that a stride of a power of two has."""
    x = torch.arange(first, first + n, device="cuda")
    return torch.tensor([-1.0, 0.0, 2.0], device="cuda")[(x % 7 + x // 11) % 3]


def _fill(t):
    for i in range(0, t.shape[0], PART):
        part = t[i:i + PART]
        part.copy_(_pattern(i, part.shape[0])[:, None].expand(part.shape))
    return t


def _check(t, value):
    """Every row of t is value(the pattern's rows there)."""
    for i in range(0, t.shape[0], PART):
        part = t[i:i + PART]
        ref = value(_pattern(i, part.shape[0]))[:, None].to(t.dtype)
        assert bool((part == ref).all()), f"rows {i} to {i + part.shape[0]}"


def test_route_and_its_gradient():
    """One expert, sigmoid scores: the weight is the score itself."""
    x = _fill(torch.empty(MOST, 1, dtype=torch.bfloat16, device="cuda"))
    keys = torch.full((MOST, 1), 7, dtype=torch.int32, device="cuda")
    w = torch.empty(MOST, 1, device="cuda")
    counts = torch.empty(1, 1, dtype=torch.int64, device="cuda")
    options = dict(score="sigmoid", renormalise=False)
    # what each of the pattern's values gets, from a call of three tokens
    three = torch.tensor([[-1.0], [0.0], [2.0]], device="cuda").bfloat16()
    k3, w3 = torch.empty(3, 1, dtype=torch.int32, device="cuda"), torch.empty(3, 1, device="cuda")
    d3 = torch.empty_like(three)
    with a2av.A2av(1) as eng:
        eng.route([three], [k3], [w3], 1, **options)
        eng.route_backward([three], [k3], [torch.ones_like(w3)], [d3], 1, **options)
        eng.route([x], [keys], [w], 1, counts=counts, **options)
        assert eng.status() == a2av.OK
        assert (w3[:, 0].cpu() - torch.sigmoid(three[:, 0].float().cpu())).abs().max() < 1e-6
        pick = lambda of: lambda v: of[:, 0].float()[torch.where(v == 2, 2, v.long() + 1)]
        assert int(counts) == MOST and not bool(keys.any())
        _check(w, pick(w3))
        d = torch.full((MOST, 1), 7.0, dtype=torch.bfloat16, device="cuda")
        w.fill_(1.0)
        eng.route_backward([x], [keys], [w], [d], 1, **options)
        assert eng.status() == a2av.OK
        _check(d, pick(d3))


@pytest.mark.parametrize("features", [1, 8])
def test_experts_forward_and_rows_gradient(features):
    """One expert, one group: rows of 16 bytes (the tensor cores) and of one
    element (plain products); ReLU, so that dz has a pass of its own."""
    D = features
    x = _fill(torch.empty(MOST, D, dtype=torch.bfloat16, device="cuda"))
    w = [(torch.eye(D, device="cuda") * 2).bfloat16().view(1, D, D)]
    counts = torch.tensor([[MOST]], device="cuda")
    y = torch.full((MOST, D), 7.0, dtype=torch.bfloat16, device="cuda")
    with a2av.A2av(1) as eng:
        eng.expert_matmul([x], counts, w, [y], activation="relu")
        assert eng.status() == a2av.OK
        _check(y, lambda v: 2 * v.clamp_min(0))
        # dy = x, pre = x (its signs): dz = x where x > 0, and twice that for the rows
        eng.expert_matmul_backward([x], counts, w, [x], d_rows=[y.fill_(7.0)], pre=[x], activation="relu")
        assert eng.status() == a2av.OK
        _check(y, lambda v: 2 * v.clamp_min(0))
    del x, y
    torch.cuda.empty_cache()


def test_a_contraction_of_more_than_a_second():
    """One expert's gradient over 2^30 rows and some: one tile, on one pair of CTAs,
    whose other waits are limited.  Products of signs: the sums are whole numbers
    that 32 bits hold exactly, so that the result is exact to its one rounding."""
    rows, D, N = (1 << 30) + 1001, 8, 8
    gen = torch.Generator("cuda").manual_seed(3)
    signs = lambda n: torch.empty(rows, n, dtype=torch.bfloat16, device="cuda").random_(
        0, 2, generator=gen).mul_(2).sub_(1)
    x, dy = signs(D), signs(N)
    w = torch.empty(1, N, D, dtype=torch.bfloat16, device="cuda")
    d_w = torch.zeros_like(w)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    with a2av.A2av(1) as eng:
        counts = torch.tensor([[rows]], device="cuda")
        begin.record()
        eng.expert_matmul_backward([x], counts, [w], [dy], d_weights=[d_w])
        end.record()
        assert eng.status() == a2av.OK
    assert begin.elapsed_time(end) > 1500, "not longer than a limited wait"
    ref = torch.zeros(N, D, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 1 << 22):  # (sums of at most 2^22 signs: exact in 32 bits)
        ref += (dy[i:i + (1 << 22)].float().T @ x[i:i + (1 << 22)].float()).double()
    assert ref.abs().max() < 2 ** 24 and torch.equal(d_w[0], ref.bfloat16())
