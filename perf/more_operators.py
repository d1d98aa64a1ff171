"""The norm before an MoE layer and microscaled rows, as cases that can be timed.

The root-mean-square norm with the residual's addition (``norm``,
``norm_backward``), packed rows of 8 or 4 bits with a scale for each 32 values
(``quantise``, ``dequantise``) and the experts' products on them
(``expert_matmul_mx``).  ``run`` computes them with elementary torch operations
in 32 bits (64 where a value next to a rounding's border, or a long sum, asks
for it), or, with ``own`` set, by the framework's calls.

A packed row of D values, Dp being D rounded up to 32: the values (e4m3: Dp
bytes; e2m1: Dp / 2, value 2 i in a byte's low half), Dp / 32 scale bytes s that
stand for 2^(s - 127), zeros up to a multiple of 32 bytes.  A block's scale is the
smallest that lets its largest value fit.

Layouts are the framework's: W ranks; rank r's tokens are a [T, ...] tensor; peer
p's rows are ordered by (source rank, local expert, token); ``counts`` [W][E] holds
the items each rank sends to each expert.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_MOST = {"mxfp8": 448.0, "mxfp4": 6.0}
_engines = {}


def _engine(W):
    """The framework's handle for W ranks; a program makes it once."""
    if W not in _engines:
        import variable_size_all_gb300 as a2av
        _engines[W] = a2av.A2av(W)
    return _engines[W]


def _value_bytes(D, fmt):
    return -(-D // 32) * (32 if fmt == "mxfp8" else 16)


def _row_bytes(D, fmt):
    return -(-(_value_bytes(D, fmt) + -(-D // 32)) // 32) * 32


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the norm of one decoding step: 4 tokens on each of 8 ranks (latency)
        {"name": "norm_decode", "op": "norm", "W": 8, "tokens": 4, "H": 7168, "dtype": "bf16",
         "residual": True, "format": "plain"},
        # the norm before the repository's MoE dispatch workload, its rows leaving in 8 bits
        {"name": "norm_moe_8bit", "op": "norm", "W": 8, "tokens": 8192, "H": 7168, "dtype": "bf16",
         "residual": True, "format": "mxfp8"},
        # its backward pass in training, the residual stream's gradient added
        {"name": "norm_backward_moe", "op": "norm_backward", "W": 8, "tokens": 8192, "H": 7168,
         "dtype": "bf16", "residual": True},
        # a short, odd batch of odd rows, which take no vectors
        {"name": "norm_backward_odd", "op": "norm_backward", "W": 2, "tokens": 777, "H": 1001,
         "dtype": "f32", "residual": False},
        # the inner activations of one decoding step, between the two products
        {"name": "quantise_decode", "op": "quantise", "W": 8, "tokens": 32, "H": 2048, "dtype": "bf16",
         "format": "mxfp8"},
        # a prompt's rows before the exchange (half the bytes to move)
        {"name": "quantise_moe", "op": "quantise", "W": 8, "tokens": 8192, "H": 7168, "dtype": "bf16",
         "format": "mxfp8"},
        # received rows, two choices a token, back in 16 bits
        {"name": "dequantise_moe", "op": "dequantise", "W": 8, "tokens": 16384, "H": 7168,
         "dtype": "bf16", "format": "mxfp8"},
        # weights through 4 bits and back: what rounding makes of 8 ranks' 2048 -> 7168
        {"name": "round_trip_4bit", "op": "round_trip", "W": 8, "tokens": 57344, "H": 2048,
         "dtype": "bf16", "format": "mxfp4"},
        # the experts of one decoding step: 16 tokens a rank, 4-bit weights (weights bound)
        {"name": "mx_decode", "op": "experts", "W": 8, "tokens": 16, "E": 64, "k": 2, "D": 7168, "N": 2048,
         "dtype": "bf16", "format": "mxfp4", "act": "silu", "gated": True, "bias": False,
         "residual": False, "skew": 0.0},
        # a prompt's second product in 8 bits, Zipf-skewed experts, ragged groups
        {"name": "mx_down", "op": "experts", "W": 8, "tokens": 1024, "E": 64, "k": 2, "D": 2048, "N": 7168,
         "dtype": "bf16", "format": "mxfp8", "act": "none", "gated": False, "bias": False,
         "residual": False, "skew": 1.2},
        # the gated product of the MoE dispatch workload's tokens, 4 bits
        {"name": "mx_up_large", "op": "experts", "W": 8, "tokens": 8192, "E": 64, "k": 2, "D": 7168,
         "N": 2048, "dtype": "bf16", "format": "mxfp4", "act": "silu", "gated": True, "bias": False,
         "residual": False, "skew": 1.2},
        # a shared (dense) layer in 8 bits: an odd number of rows, every part of the epilogue
        {"name": "mx_linear", "op": "experts", "W": 1, "tokens": 5001, "E": 1, "k": 1, "D": 7168, "N": 2048,
         "dtype": "f16", "format": "mxfp8", "act": "gelu", "gated": False, "bias": True,
         "residual": True, "skew": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "norm_backward", "quantise", "dequantise",
                     "round_trip", "experts", "experts", "experts", "experts"])
    W = rng.choice([1, 2, 4, 8])
    fmt = rng.choice(["mxfp8", "mxfp4"])
    width = _log_int(rng, 33, 7168) if rng.random() < 0.4 else 32 * _log_int(rng, 1, 224)
    if op != "experts":
        # (the norm's 4-bit output is a round trip's rounding of the norm's)
        return {"op": op, "W": W, "tokens": _log_int(rng, 1, 8192), "H": width,
                "dtype": rng.choice(["bf16", "f16", "f32"]),
                **({"format": rng.choice(["plain", "mxfp8"])} if op == "norm" else
                   {"format": "mxfp8" if op == "quantise" else "mxfp4" if op == "round_trip" else fmt}
                   if op != "norm_backward" else {}),
                **({"residual": rng.random() < 0.6} if op.startswith("norm") else {})}
    E = W * _log_int(rng, 1, 64 // W)
    k = rng.randint(1, min(4, E))
    gated = rng.random() < 0.5
    N = _log_int(rng, 33, 7168) if rng.random() < 0.3 else 8 * _log_int(rng, 8, 896)
    if gated or E > 32:
        N = min(N, 2048)
    rows = 131072 * 2048 // max(2048, N)
    return {"op": op, "W": W, "tokens": max(1, min(_log_int(rng, 1, 8192), rows // (W * k))), "E": E,
            "k": k, "D": width, "N": N, "dtype": rng.choice(["bf16", "f16"]), "format": fmt,
            "act": rng.choice(["relu", "gelu", "silu"] if gated else ["none", "relu", "gelu", "silu"]),
            "gated": gated, "bias": rng.random() < 0.5, "residual": rng.random() < 0.3,
            "skew": rng.choice([0.0, 0.8, 1.2])}


# ----------------------------------------------------------------- inputs --
def _popularity(case, device):
    """Experts' popularity: k^-skew, spread over the expert ids by a fixed stride."""
    E = case["E"]
    place = torch.arange(E, device=device, dtype=torch.float32)
    place = (place * 29 + 7) % E if E % 29 else place
    return (place + 1) ** -case["skew"]


def _routed(case, gen):
    """counts [W, E] of a routing by popularity, and the rows each peer holds."""
    W, T, E, k = case["W"], case["tokens"], case["E"], case["k"]
    u = torch.rand((W, T, E), generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)
    choices = (_popularity(case, "cuda").log() - (-u.log()).log()).topk(k, dim=-1).indices
    counts = torch.zeros((W, E), dtype=torch.int64, device="cuda")
    counts.scatter_add_(1, choices.reshape(W, T * k), torch.ones((W, T * k), dtype=torch.int64, device="cuda"))
    return counts, counts.view(W, W, E // W).sum((0, 2)).tolist()


def _normal(shape, gen, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _hidden(shape, gen, dtype):
    """Rows of a residual stream: channels of different spread."""
    spread = torch.exp(0.5 * torch.randn(shape[-1], generator=gen, device="cuda"))
    return (torch.randn(shape, generator=gen, device="cuda") * spread).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * int(seed) + 29)
    W, T, op = case["W"], case["tokens"], case["op"]
    dt = _DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if op == "experts":
        D, N, E, fmt = case["D"], case["N"], case["E"], case["format"]
        K, Z = E // W, 2 * N if case["gated"] else N
        counts, rows = _routed(case, gen)
        M = W * T * case["k"]
        s["counts"] = counts
        s["rows"] = torch.empty((M, _row_bytes(D, fmt)), dtype=torch.uint8, device="cuda")
        for at in range(0, M, 32768):
            part = s["rows"][at:at + 32768]
            part.copy_(_pack(_normal((part.shape[0], D), gen, dt).float(), fmt))
        s["weights"] = torch.empty((E, Z, _row_bytes(D, fmt)), dtype=torch.uint8, device="cuda")
        for e in range(E):
            s["weights"][e] = _pack(_normal((Z, D), gen, dt, D ** -0.5).float(), fmt)
        s["rows_of"], s["weights_of"] = list(s["rows"].split(rows)), list(s["weights"].view(W, K, Z, -1))
        s["bias"] = _normal((E, Z), gen, dt, 0.2) if case["bias"] else None
        s["bias_of"] = list(s["bias"].view(W, K, Z)) if case["bias"] else None
        s["residual"] = _normal((M, N), gen, dt) if case["residual"] else None
        s["residual_of"] = list(s["residual"].split(rows)) if case["residual"] else None
        s["out"] = torch.empty((M, N), dtype=dt, device="cuda")
        s["out_of"] = list(s["out"].split(rows))
        return s
    H, fmt = case["H"], case.get("format")
    new = lambda dtype, width=H: torch.empty((W * T, width), dtype=dtype, device="cuda")
    if op == "dequantise":
        s["packed"] = torch.empty((W * T, _row_bytes(H, fmt)), dtype=torch.uint8, device="cuda")
        for at in range(0, W * T, 32768):
            part = s["packed"][at:at + 32768]
            part.copy_(_pack(_hidden((part.shape[0], H), gen, dt).float(), fmt))
        s["packed_of"] = list(s["packed"].split(T))
        s["out"] = new(dt)
        s["out_of"] = list(s["out"].split(T))
        return s
    s["x"] = _hidden((W * T, H), gen, dt)
    s["x_of"] = list(s["x"].split(T))
    if op in ("quantise", "round_trip"):
        s["packed"] = new(torch.uint8, _row_bytes(H, fmt))
        s["packed_of"] = list(s["packed"].split(T))
        s["out"] = new(dt) if op == "round_trip" else None
        s["out_of"] = list(s["out"].split(T)) if op == "round_trip" else None
        return s
    s["weight"] = 1 + 0.1 * torch.randn(H, generator=gen, device="cuda")
    if op == "norm":
        s["residual"] = _hidden((W * T, H), gen, dt) if case["residual"] else None
        s["residual_of"] = list(s["residual"].split(T)) if case["residual"] else None
        s["sums_of"] = list(new(dt).split(T)) if case["residual"] else None
        s["out"] = new(dt) if fmt == "plain" else new(torch.uint8, _row_bytes(H, fmt))
        s["out_of"] = list(s["out"].split(T))
        return s
    # (x is what the forward pass kept: the sums)
    s["d_out"] = _normal((W * T, H), gen, dt)
    s["d_out_of"] = list(s["d_out"].split(T))
    s["d_sums"] = _normal((W * T, H), gen, dt) if case["residual"] else None
    s["d_sums_of"] = list(s["d_sums"].split(T)) if case["residual"] else None
    s["d_x_of"] = list(new(dt).split(T))
    s["d_weight"] = torch.empty(H, device="cuda")
    return s


_EPS = 1e-6

# ------------------------------------------------------------ plain forms --
def _blocks(x):
    """[rows, D] as [rows, blocks, 32], zeros behind."""
    D = x.shape[1]
    Dp = -(-D // 32) * 32
    if Dp != D:
        x = torch.cat([x, x.new_zeros((x.shape[0], Dp - D))], 1)
    return x.view(x.shape[0], Dp // 32, 32)


def _scaled(x, fmt):
    """Blocks divided by their scales, and the scales' bytes."""
    x = _blocks(x)
    m, e = torch.frexp(x.abs().amax(-1) / _MOST[fmt])  # m 2^e, m in [0.5, 1)
    s = (torch.where(m > 0.5, e, e - 1) + 127).clamp(0, 254)
    s = torch.where(m == 0, torch.zeros_like(s), s)
    return x * torch.exp2((127 - s).to(x.dtype))[..., None], s


def _codes4(v):
    """The 4-bit codes of e2m1, nearest, ties to the even code."""
    a = v.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
         + (a > 5.0))
    return c + 8 * (v < 0).to(torch.uint8)


def _pack(x, fmt):
    """Packed rows of [rows, D] values."""
    D = x.shape[1]
    v, s = _scaled(x, fmt)
    v = v.reshape(x.shape[0], -1)
    if fmt == "mxfp8":
        codes = v.float().to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        codes = _codes4(v)
        codes = codes[:, 0::2] + 16 * codes[:, 1::2]
    rows = torch.cat([codes, s.to(torch.uint8)], 1)
    fill = _row_bytes(D, fmt) - rows.shape[1]
    return torch.cat([rows, rows.new_zeros((rows.shape[0], fill))], 1) if fill else rows


def _unpack(rows, D, fmt):
    """The values of packed rows, in 32 bits."""
    V, B = _value_bytes(D, fmt), -(-D // 32)
    if fmt == "mxfp8":
        v = rows[:, :V].contiguous().view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=rows.device)
        table = torch.cat([table, -table])
        b = rows[:, :V].long()
        v = torch.stack([table[b & 15], table[b >> 4]], -1)
    s = torch.exp2(rows[:, V:V + B].float() - 127)
    return (v.reshape(rows.shape[0], B, 32) * s[..., None]).reshape(rows.shape[0], -1)[:, :D]


def _parts(rows, D, fmt):
    """What 8-bit rows hold, as the types whose values it stands for: views."""
    V, B = _value_bytes(D, fmt), -(-D // 32)
    return {"values": rows[:, :D].view(torch.float8_e4m3fn),
            "scales": rows[:, V:V + B].view(torch.float8_e8m0fnu)}


def _plain_norm(s):
    case, x = s["case"], s["x"]
    plain = case["format"] == "plain"
    # (the sums are rounded to the rows' type, and the norm is theirs)
    t = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    v = t.float() if plain else t.double()
    y = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + _EPS) * s["weight"].to(v.dtype)
    sums = None if s["residual"] is None else t
    if plain:
        return {"out": y.to(x.dtype), "sums": sums}
    return {**_parts(_pack(y, case["format"]), case["H"], case["format"]), "sums": sums}


def _plain_norm_backward(s):
    dt = s["x"].dtype
    v, dy = s["x"].float(), s["d_out"].float()
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + _EPS)
    g = dy * s["weight"]
    d = r * (g - v * (r * r * (g * v).mean(-1, keepdim=True)))
    if s["d_sums"] is not None:
        d = d + s["d_sums"].float()
    return {"d_x": d.to(dt), "d_weight": (dy * v * r).sum(0, dtype=torch.float64).float()}


def _plain_quantise(s):
    case = s["case"]
    return _parts(_pack(s["x"].float(), case["format"]), case["H"], case["format"])


def _plain_dequantise(s):
    case = s["case"]
    return {"out": _unpack(s["packed"], case["H"], case["format"]).to(s["out"].dtype)}


def _plain_round_trip(s):
    case = s["case"]
    return {"out": _unpack(_pack(s["x"].float(), case["format"]), case["H"], case["format"]).to(s["x"].dtype)}


def _groups(case, counts):
    """(expert, its segments [start, end) of the rows of all peers): the order is (peer, source, expert)."""
    W, K = case["W"], case["E"] // case["W"]
    seg = counts.view(W, W, K).permute(1, 0, 2).reshape(-1)
    end = seg.cumsum(0).tolist()
    start = [0] + end[:-1]
    for p in range(W):
        for e in range(K):
            at = [(p * W + r) * K + e for r in range(W)]
            yield p * K + e, [(start[i], end[i]) for i in at if end[i] > start[i]]


def _act(case, z):
    a = case["act"]
    if a == "relu":
        return z.clamp_min(0)
    if a == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if a == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _plain_experts(s):
    case = s["case"]
    D, N, fmt = case["D"], case["N"], case["format"]
    out = torch.empty_like(s["out"])
    for e, segments in _groups(case, s["counts"]):
        if not segments:
            continue
        at = torch.cat([torch.arange(a, b, device=out.device) for a, b in segments])
        z = _unpack(s["rows"][at], D, fmt) @ _unpack(s["weights"][e], D, fmt).T
        if s["bias"] is not None:
            z = z + s["bias"][e].float()
        y = _act(case, z[:, :N]) * z[:, N:] if case["gated"] else _act(case, z)
        if s["residual"] is not None:
            y = y + s["residual"][at].float()
        out[at] = y.to(out.dtype)
    return {"out": out}


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "quantise": _plain_quantise,
          "dequantise": _plain_dequantise, "round_trip": _plain_round_trip, "experts": _plain_experts}


# ---------------------------------------------------------- the framework --
def _own_norm(s):
    c = s["case"]
    fmt = None if c["format"] == "plain" else c["format"]
    _engine(c["W"]).norm(s["x_of"], s["weight"], s["out_of"], residual=s["residual_of"],
                         sums=s["sums_of"], eps=_EPS, format=fmt)
    sums = None if s["residual"] is None else s["sums_of"][0]._base
    return {"sums": sums, **({"out": s["out"]} if fmt is None else _parts(s["out"], c["H"], fmt))}


def _own_norm_backward(s):
    _engine(s["case"]["W"]).norm_backward(s["x_of"], s["weight"], s["d_out_of"], s["d_x_of"],
                                          d_weight=s["d_weight"], d_sums=s["d_sums_of"], eps=_EPS)
    return {"d_x": s["d_x_of"][0]._base, "d_weight": s["d_weight"]}


def _own_quantise(s):
    c = s["case"]
    _engine(c["W"]).quantise(s["x_of"], s["packed_of"], c["format"])
    return _parts(s["packed"], c["H"], c["format"])


def _own_dequantise(s):
    c = s["case"]
    _engine(c["W"]).dequantise(s["packed_of"], s["out_of"], c["format"])
    return {"out": s["out"]}


def _own_round_trip(s):
    c = s["case"]
    _engine(c["W"]).quantise(s["x_of"], s["packed_of"], c["format"])
    _engine(c["W"]).dequantise(s["packed_of"], s["out_of"], c["format"])
    return {"out": s["out"]}


def _own_experts(s):
    c = s["case"]
    _engine(c["W"]).expert_matmul_mx(s["rows_of"], s["counts"], s["weights_of"], s["out_of"], c["D"],
                                     c["format"], activation=c["act"], gated=c["gated"],
                                     bias=s["bias_of"], residual=s["residual_of"])
    return {"out": s["out"]}


_OWN = {"norm": _own_norm, "norm_backward": _own_norm_backward, "quantise": _own_quantise,
        "dequantise": _own_dequantise, "round_trip": _own_round_trip, "experts": _own_experts}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------- work --
def work(case):
    W, T, op = case["W"], case["tokens"], case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    if op != "experts":
        H, rows, fmt = case["H"], W * T, case.get("format")
        whole = rows * H * size
        if op == "norm":
            out = whole if fmt == "plain" else rows * _row_bytes(H, fmt)
            return {"bytes": whole * (3 if case["residual"] else 1) + out + 4 * H, "flops": 4 * rows * H}
        if op == "norm_backward":
            return {"bytes": whole * (4 if case["residual"] else 3) + 8 * H, "flops": 10 * rows * H}
        packed = rows * _row_bytes(H, fmt)
        if op == "round_trip":
            return {"bytes": 2 * (whole + packed), "flops": 4 * rows * H}
        return {"bytes": whole + packed, "flops": 2 * rows * H}
    D, N, E = case["D"], case["N"], case["E"]
    items, Z, row = W * T * case["k"], 2 * N if case["gated"] else N, _row_bytes(D, case["format"])
    pop = _popularity(case, "cpu").double()
    hit = float((1 - (1 - pop / pop.sum()) ** items).sum())  # experts with a row, on average
    return {"bytes": items * (row + N * size * (2 if case["residual"] else 1)) + hit * Z * row + W * E * 8,
            "flops": 2.0 * items * D * Z}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The definitions in 64 bits."""
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "quantise": _exact_quantise,
            "dequantise": _exact_dequantise, "round_trip": _exact_quantise,
            "experts": _exact_experts}[case["op"]](case, prepare(case, seed))


def _grid(v, fmt):
    """The nearest value that a code holds (ties to the even one): the step follows the exponent."""
    least, digits = (-6, 3) if fmt == "mxfp8" else (0, 1)
    e = torch.log2(v.abs().clamp_min(2.0 ** -300)).floor().clamp_min(least)
    step = torch.exp2(e - digits)
    return (v / step).round() * step


def _exact_rounded(y, fmt):
    """(codes' values, scales) of 64-bit rows."""
    rows, D = y.shape
    pad = (-D) % 32
    y = torch.nn.functional.pad(y, (0, pad)).unflatten(1, (-1, 32))
    largest = y.abs().max(dim=2).values
    e = torch.log2(largest / _MOST[fmt]).ceil()
    e = torch.where(largest > _MOST[fmt] * torch.exp2(e), e + 1, e)  # (where the logarithm was rounded)
    e = torch.where(largest <= _MOST[fmt] * torch.exp2(e - 1), e - 1, e).clamp(-127, 127)
    scale = torch.exp2(e)
    return _grid(y / scale[:, :, None], fmt).reshape(rows, -1)[:, :D], scale


def _exact_norm(case, s):
    x = s["x"].double()
    sums = None
    if s["residual"] is not None:
        sums = x + s["residual"].double()
        # (the norm is defined on the sums as they are kept)
        x = sums.float().to(s["x"].dtype).double()
    y = x / (x.square().sum(1, keepdim=True) / x.shape[1] + _EPS).sqrt() * s["weight"].double()
    if case["format"] == "plain":
        return {"out": y, "sums": sums}
    values, scales = _exact_rounded(y, case["format"])
    return {"values": values, "scales": scales, "sums": sums}


def _exact_norm_backward(case, s):
    """Through the unit row: y = w * u, u = x / |x|_rms."""
    H = case["H"]
    x, dy = s["x"].double(), s["d_out"].double()
    rms = (x.square().sum(1, keepdim=True) / H + _EPS).sqrt()
    u = x / rms
    du = dy * s["weight"].double()
    d = (du - u * (du * u).sum(1, keepdim=True) / H) / rms
    if s["d_sums"] is not None:
        d += s["d_sums"].double()
    return {"d_x": d, "d_weight": torch.einsum("th,th->h", dy, u)}


def _exact_quantise(case, s):
    values, scales = _exact_rounded(s["x"].double(), case["format"])
    if case["op"] == "quantise":
        return {"values": values, "scales": scales}
    return {"out": values * scales.repeat_interleave(32, 1)[:, :case["H"]]}


def _exact_values(rows, D, fmt):
    """Packed rows from their bits: sign, exponent and digits of each code, in 64 bits."""
    V = _value_bytes(D, fmt)
    codes = rows[:, :V].to(torch.int32)
    if fmt == "mxfp8":
        sign, e, m, bias, digits = codes >> 7, (codes >> 3) & 15, codes & 7, 7, 3
    else:
        codes = torch.stack([codes & 15, codes >> 4], 2).flatten(1)
        sign, e, m, bias, digits = codes >> 3, (codes >> 1) & 3, codes & 1, 1, 1
    m = m.double() / 2 ** digits
    v = torch.where(e == 0, m * 2.0 ** (1 - bias), torch.ldexp(1 + m, e - bias))
    v = torch.where(sign == 1, -v, v)[:, :D]
    scale = torch.ldexp(torch.ones((), dtype=torch.float64, device=rows.device),
                        rows[:, V:V + -(-D // 32)].to(torch.int32) - 127)
    return v * scale.repeat_interleave(32, 1)[:, :D]


def _exact_dequantise(case, s):
    rows = s["packed"]
    return {"out": torch.cat([_exact_values(r, case["H"], case["format"]) for r in rows.split(16384)])}


def _exact_experts(case, s):
    W, K, D, N, fmt = case["W"], case["E"] // case["W"], case["D"], case["N"], case["format"]
    if 2.0 * W * case["tokens"] * case["k"] * D * N * (2 if case["gated"] else 1) > 1.2e13:
        return None  # (64-bit products of more than some 20 seconds)
    counts = s["counts"].cpu().numpy()
    outs = []
    for p in range(W):
        rows, weights = s["rows_of"][p], s["weights_of"][p]
        # the expert of each row of this peer: (source, local expert) in order
        owner = torch.from_numpy(np.tile(np.arange(K), W).repeat(counts[:, p * K:(p + 1) * K].reshape(-1))).cuda()
        out = torch.zeros((rows.shape[0], N), dtype=torch.float64, device="cuda")
        for e in range(K):
            at = (owner == e).nonzero().reshape(-1)
            z = torch.einsum("md,nd->mn", _exact_values(rows[at], D, fmt), _exact_values(weights[e], D, fmt))
            if s["bias"] is not None:
                z += s["bias_of"][p][e].double()
            g = z[:, :N]
            y = {"none": lambda: g, "relu": lambda: torch.relu(g), "silu": lambda: g * torch.sigmoid(g),
                 "gelu": lambda: g * 0.5 * torch.erfc(-g * 0.5 ** 0.5)}[case["act"]]()
            if case["gated"]:
                y = y * z[:, N:]
            if s["residual"] is not None:
                y = y + s["residual_of"][p][at].double()
            out[at] = y
        outs.append(out)
    return {"out": torch.cat(outs)}
