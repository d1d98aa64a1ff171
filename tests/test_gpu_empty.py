"""The weighted combine of an empty batch: no token on any rank."""
import pytest
import torch

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()


@pytest.mark.parametrize("module", ["_marshal", "_PlainMarshal"])
@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("W,k", [(1, 2), (4, 3), (2, 1)])
def test_no_tokens_on_any_rank(W, k, flat, module):
    """An empty batch: nothing to sum, and weights of [0, k] are what belongs to it."""
    new = lambda dtype, *shape: [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(W)]
    keys = new(torch.int32, 0) if flat else new(torch.int32, 0, k)
    pos, rows, y = new(torch.int64, 0), new(torch.bfloat16, 5, 16), new(torch.bfloat16, 0, 16)
    w, d_w = new(torch.float32, 0, k), new(torch.float32, 0, k)
    d_rows = [torch.full_like(t, 7) for t in rows]
    S = torch.zeros(W, W, dtype=torch.int64, device="cuda")
    with a2av.A2av(W) as eng:
        eng._marshal = getattr(a2av, module)
        for weights in (w, None):
            eng.combine_weighted(rows, S, keys, pos, 2, weights, y, residual=y)
            eng.bind_combine_weighted(rows, S, keys, pos, 2, weights, y)()
            eng.combine_weighted_backward(rows, S, keys, pos, 2, weights, y, d_rows, d_w)
            eng.combine_weighted_backward(None, S, keys, pos, 2, weights, y, d_rows)
        assert eng.status() == a2av.OK
        with pytest.raises(ValueError):
            eng.combine_weighted(rows, S, keys, pos, 2, new(torch.float32, 1, k), y)
        if not flat and k > 1:
            with pytest.raises(ValueError):
                eng.combine_weighted(rows, S, keys, pos, 2, new(torch.float32, 0, k + 1), y)
    assert all((t == 7).all() for t in d_rows)
