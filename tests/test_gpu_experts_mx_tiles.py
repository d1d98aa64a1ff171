"""The experts' products on packed rows where every pair of CTAs takes several tiles
of several stages, against the definition in 64 bits: the scales of one tile are on
their way while the last one's are in use."""
import pytest
import torch

from tests import test_gpu_experts_mx as products

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()


# values of a row: pieces of 16 scales (512 values) 1, 2 (the second of one block, of some,
# full), 3 and 4, stages of 128 or 256 values whole and not
@pytest.mark.parametrize("D", [288, 544, 600, 1000, 1056, 2048])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_several_tiles_a_pair(fmt, gated, D):
    """24 experts of 1280 features, about 180 rows each: 170 tiles and more for 76 pairs (twice
    that gated), of one or two rows of tiles."""
    c = products._case(2, 12, D, 1280, 90, "bf16", fmt, gated, seed=D, slack=5)
    name = "silu" if gated else "none"
    out = products._run(c, name, True, False)
    products._check(c, name, True, False, out)
    for _ in range(3):
        again = products._run(c, name, True, False)
        assert all(torch.equal(a, b) for a, b in zip(again, out))


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_counts_of_any_alignment(fmt):
    """Counts eight bytes off sixteen, with tiles that have fewer rows and features than places."""
    c = products._case(2, 3, 96, 40, 9, "bf16", fmt, False, seed=12, slack=2)
    want = products._run(c, "relu", True, False)
    counts = torch.empty(c["d_counts"].numel() + 1, dtype=torch.int64, device="cuda")[1:].view(c["d_counts"].shape)
    counts.copy_(c["d_counts"])
    assert counts.data_ptr() % 16 == 8
    c["d_counts"] = counts
    assert all(torch.equal(a, b) for a, b in zip(products._run(c, "relu", True, False), want))
