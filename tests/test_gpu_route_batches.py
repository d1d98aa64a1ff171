"""The router's choices and weights of a token do not depend on its batch."""
import pytest
import torch

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()


@pytest.mark.parametrize("E", [8, 24, 60, 64, 100, 256])
@pytest.mark.parametrize("options", [dict(renormalise=False), dict(renormalise=True),
                                     dict(score="sigmoid", renormalise=True),
                                     dict(groups=4, top_groups=2, group_top=2, renormalise=False)], ids=str)
@pytest.mark.parametrize("with_bias", [False, True])
def test_a_token_is_routed_the_same_in_any_batch(E, options, with_bias):
    """Few tokens and many take different forms of the kernel: the same keys, and
    the same weights to the bit, for a token in a prompt and in a decoding step."""
    gen = torch.Generator("cuda").manual_seed(E)
    x = torch.randn(3000, E, device="cuda", generator=gen) * 2
    bias = torch.randn(E, device="cuda", generator=gen) * 0.01 if with_bias else None
    k = min(7, E // 4 * options.get("top_groups", 4))
    if options.get("groups", 1) > 1 and E // 4 < 2:
        pytest.skip("groups of two choices")
    results = []
    with a2av.A2av(1) as eng:
        for batch in (3000, 250):
            keys = torch.empty(3000, k, dtype=torch.int32, device="cuda")
            w = torch.empty(3000, k, device="cuda")
            for t in range(0, 3000, batch):
                eng.route([x[t:t + batch]], [keys[t:t + batch]], [w[t:t + batch]], k, bias=bias, **options)
            assert eng.status() == a2av.OK
            results.append((keys, w))
    (a, v), (b, w) = results
    assert torch.equal(a, b) and torch.equal(v, w)
