"""The MoE operators' calls, made whole by the compiled module (csrc/marshal.cpp),
against the same calls made argument by argument: equal results, also on a
stream of the caller's and with a rank without tokens; and what the module does
not take is refused, or done, as the methods themselves do."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()


class _Counting:
    """A module's functions, with the number of calls that were made whole."""

    def __init__(self, module):
        self._module, self.whole = module, 0

    def __getattr__(self, name):
        f = getattr(self._module, name)

        def counted(*args):
            result = f(*args)
            if name in ("route", "route_backward", "expert_matmul", "expert_matmul_backward",
                        "combine_weighted", "combine_weighted_backward") and result is not None:
                self.whole += 1
            return result
        return counted


def _layer(plain, shape=(2, 33, 64, 48, 6, 2), dtype=torch.bfloat16):
    from moe_layer import MoeLayer
    torch.manual_seed(0)
    layer = MoeLayer(*shape, dtype=dtype)
    # (never a module that was not built: the compiled one has to be there)
    layer.engine._marshal = _Counting(a2av._PlainMarshal if plain else a2av._marshal)
    return layer


@pytest.fixture(scope="module", autouse=True)
def _compiled(_cuda):
    import variable_size_all_gb300._marshal  # noqa: F401


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_layer_is_the_same(side, dtype):
    results = []
    for plain in (False, True):
        layer = _layer(plain, dtype=dtype)
        x = [torch.randn(layer.T, layer.H, device="cuda").to(dtype) for _ in range(layer.W)]
        dy = [torch.randn_like(t) for t in x]
        stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            y, dx = layer.forward(x), layer.backward(dy)
        stream.synchronize()
        assert layer.engine.status() == a2av.OK
        # route, two products, combine; combine's gradient, the dispatch's, route's, and one
        # product's: the first, and the second if it needs more, make the workspace first
        assert layer.engine._marshal.whole in ((0,) if plain else (7, 8))
        if not plain:
            with torch.cuda.stream(stream):
                layer.backward(dy)
            stream.synchronize()
            assert layer.engine._marshal.whole in (12, 13)
        results.append([t.clone() for t in [*y, *dx, *layer.keys, *layer.weights, layer.counts,
                                            *layer.d_up, *layer.d_down, layer.d_gate]])
        layer.engine.close()
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_options_are_the_same():
    """Every option of each call, on a given stream, with a rank without tokens."""
    results = []
    W, E, k, H, N, T = 4, 16, 3, 64, 32, (5, 0, 17, 8)
    stream = torch.cuda.Stream()
    for module in (a2av._marshal, a2av._PlainMarshal):
        torch.manual_seed(2)
        new = lambda widths, dtype: [torch.zeros(t, widths, dtype=dtype, device="cuda") for t in T]
        logits = [torch.randn(t, E, device="cuda").half() for t in T]
        bias = torch.randn(E, device="cuda")
        keys, weights = new(k, torch.int32), new(k, torch.float32)
        counts = torch.zeros(W, E, dtype=torch.int64, device="cuda")
        up = [torch.randn(E // W, 2 * N, H, device="cuda").half() for _ in T]
        b = [torch.randn(E // W, 2 * N, device="cuda").half() for _ in T]
        with a2av.A2av(W) as eng:
            eng._marshal = _Counting(module)
            stream.wait_stream(torch.cuda.current_stream())
            options = dict(score="sigmoid", renormalise=False, scale=2, stream=stream)
            eng.route(logits, keys, weights, k, counts=counts, bias=bias, groups=4, top_groups=2,
                      group_top=2, **options)
            d_logits = [torch.empty_like(t) for t in logits]
            stream.wait_stream(torch.cuda.current_stream())
            eng.route_backward(logits, keys, weights, d_logits, k, **options)
            stream.synchronize()
            held = counts.view(W, W, -1).sum((0, 2)).tolist()
            splits = counts.view(W, W, -1).sum(2)
            rows = [torch.randn(m, H, device="cuda").half() for m in held]
            res = [torch.randn(m, N, device="cuda").half() for m in held]
            out = [torch.empty_like(t) for t in res]
            pre = [torch.empty(m, 2 * N, device="cuda").half() for m in held]
            stream.wait_stream(torch.cuda.current_stream())
            eng.expert_matmul(rows, counts, up, out, activation="gelu", gated=True, bias=b, residual=res,
                              pre=pre, stream=stream)
            # an item's position: how many of its rank's items come before it in the order of keys
            pos = [torch.argsort(torch.argsort(q.view(-1), stable=True)) for q in keys]
            y, r = new(N, torch.float16), [torch.randn(t, N, device="cuda").half() for t in T]
            d_out, d_w = [torch.empty_like(t) for t in out], new(k, torch.float32)
            stream.wait_stream(torch.cuda.current_stream())
            eng.combine_weighted(out, splits, keys, pos, E // W, weights, y, residual=r, stream=stream)
            eng.combine_weighted_backward(out, splits, keys, pos, E // W, weights, r, d_out, d_w,
                                          stream=stream)
            eng.combine_weighted_backward(None, splits, keys, pos, E // W, None, y, d_peers=rows_like(out),
                                          stream=stream)
            stream.synchronize()
            assert eng.status() == a2av.OK
            assert eng._marshal.whole == (6 if module is a2av._marshal else 0)
            d_rows, d_up, d_b = rows_like(rows), rows_like(up), rows_like(b)
            need = a2av.a2av_expert_matmul_workspace_bytes(
                W, a2av.A2avExpert(E // W, H, N, a2av.F16, 2, 1), sum(held))
            space = torch.empty(need, dtype=torch.uint8, device="cuda")
            stream.wait_stream(torch.cuda.current_stream())
            for given in (dict(d_rows=d_rows, d_bias=d_b), dict(d_weights=d_up)):
                eng.expert_matmul_backward(rows, counts, up, res, pre=pre, activation="gelu", gated=True,
                                           workspace=space, stream=stream, **given)
            stream.synchronize()
            assert eng.status() == a2av.OK
            assert eng._marshal.whole == (8 if module is a2av._marshal else 0)
            with pytest.raises(a2av.A2avError):  # (a workspace that is too small)
                eng.expert_matmul_backward(rows, counts, up, res, d_rows, pre=pre, activation="gelu",
                                           gated=True, workspace=space[:need - 256])
            results.append([*keys, *weights, counts, *d_logits, *out, *pre, *y, *d_out, *d_w, *d_rows,
                            *d_up, *d_b])
    for a, c in zip(*results):
        assert torch.equal(a, c)


def rows_like(tensors):
    return [torch.empty_like(t) for t in tensors]


def test_refusals_and_missing_tensors():
    logits = [torch.randn(4, 8, device="cuda"), torch.randn(3, 8, device="cuda")]
    keys = [torch.empty(t.shape[0], 2, dtype=torch.int32, device="cuda") for t in logits]
    weights = [torch.empty(t.shape[0], 2, device="cuda") for t in logits]
    good = dict(logits=logits, keys=keys, weights=weights, topk=2)
    eng = a2av.A2av(2)
    for change in (dict(logits=logits[:1]), dict(logits=[t.double() for t in logits]),
                   dict(keys=[t.long() for t in keys]), dict(keys=keys[::-1]), dict(topk=9),
                   dict(topk=3), dict(weights=[t.t() for t in weights]), dict(score="tanh"),
                   dict(bias=torch.zeros(7, device="cuda")), dict(bias=torch.zeros(8)),
                   dict(counts=torch.zeros(2, 7, dtype=torch.int64, device="cuda")),
                   dict(logits=[t.cpu() for t in logits])):
        with pytest.raises(ValueError):
            eng.route(**{**good, **change})
    with pytest.raises(a2av.A2avError) as e:  # (the library's own refusal)
        eng.route(**good, groups=3)
    assert e.value.code == a2av.ERR_INVALID_ARG
    # a rank without a buffer, which the module leaves to the method
    eng.route([logits[0], None], [keys[0], None], [weights[0], None], 2)
    first = keys[0].clone()
    eng.route(**good)
    assert torch.equal(first, keys[0]) and eng.status() == a2av.OK
    eng.close()
    with pytest.raises(Exception):  # (a closed handle)
        eng.route(**good)
