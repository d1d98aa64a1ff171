"""The operators of an MoE layer around the exchange, as cases that can be timed.

Three operators, each with its backward pass: the router (``route``), the
experts' products (``expert_matmul``) and the weighted return path
(``combine_weighted``).  ``run`` computes them with elementary torch
operations in 32 bits, or, with ``own`` set, by the framework's calls.

Layouts are the framework's: W ranks; rank r's tokens are a [T_r, ...] tensor;
peer p's rows are ordered by (source rank, local expert, token); ``counts``
[W][E] holds the items each rank sends to each expert.  The peers' buffers
are views, one after the other, of one allocation, which is what ``run``
returns: how many rows each peer holds depends on the routing, their sum
does not.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_engines = {}


def _engine(W):
    """The framework's handle for W ranks; a program makes it once."""
    if W not in _engines:
        import variable_size_all_gb300 as a2av
        _engines[W] = a2av.A2av(W)
    return _engines[W]


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decoding step's routing: 4 tokens on each of 8 ranks (latency)
        {"name": "route_decode", "op": "route", "W": 8, "tokens": 4, "E": 64, "k": 2, "dtype": "f32",
         "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_top": 1,
         "renormalise": True, "scale": 1.0},
        # the routing of the repository's MoE dispatch workload: 8192 tokens a rank, top 2 of 64
        {"name": "route_moe", "op": "route", "W": 8, "tokens": 8192, "E": 64, "k": 2, "dtype": "bf16",
         "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_top": 1,
         "renormalise": True, "scale": 1.0},
        # many small experts: sigmoid scores, balance bias, 4 of 8 groups, top 8 of 256
        {"name": "route_grouped", "op": "route", "W": 8, "tokens": 8192, "E": 256, "k": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_top": 2,
         "renormalise": True, "scale": 2.5},
        # the router's backward pass, dense in the logits (softmax over all experts)
        {"name": "route_backward", "op": "route_backward", "W": 8, "tokens": 8192, "E": 256, "k": 8,
         "dtype": "f32", "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_top": 1,
         "renormalise": False, "scale": 1.0},
        # the experts of one decoding step: 16 tokens a rank, a row or two for each expert (weights bound)
        {"name": "experts_decode", "op": "experts", "W": 8, "tokens": 16, "E": 64, "k": 2, "D": 7168,
         "N": 2048, "dtype": "bf16", "act": "silu", "gated": True, "bias": False, "residual": False,
         "skew": 0.0},
        # a prompt's second product (back to the hidden size), Zipf-skewed experts, ragged groups
        {"name": "experts_down", "op": "experts", "W": 8, "tokens": 1024, "E": 64, "k": 2, "D": 2048,
         "N": 7168, "dtype": "bf16", "act": "none", "gated": False, "bias": False, "residual": False,
         "skew": 1.2},
        # the first, gated product of a full training batch (the MoE dispatch workload's tokens)
        {"name": "experts_up_large", "op": "experts", "W": 8, "tokens": 8192, "E": 64, "k": 2, "D": 7168,
         "N": 2048, "dtype": "bf16", "act": "silu", "gated": True, "bias": False, "residual": False,
         "skew": 1.2},
        # a shared (dense) layer: one expert, an odd number of rows, every part of the epilogue
        {"name": "linear_residual", "op": "experts", "W": 1, "tokens": 5001, "E": 1, "k": 1, "D": 2048,
         "N": 7168, "dtype": "f16", "act": "gelu", "gated": False, "bias": True, "residual": True,
         "skew": 0.0},
        # the backward pass of the gated product in training
        {"name": "experts_backward", "op": "experts_backward", "W": 8, "tokens": 2048, "E": 64, "k": 2,
         "D": 7168, "N": 2048, "dtype": "bf16", "act": "silu", "gated": True, "bias": True,
         "residual": False, "skew": 1.2},
        # the return path of one decoding step
        {"name": "combine_decode", "op": "combine", "W": 8, "tokens": 16, "E": 64, "k": 2, "H": 7168,
         "dtype": "bf16", "residual": True, "skew": 1.2},
        # the return path of a full batch
        {"name": "combine_moe", "op": "combine", "W": 8, "tokens": 8192, "E": 64, "k": 2, "H": 7168,
         "dtype": "bf16", "residual": False, "skew": 1.2},
        # and its backward pass
        {"name": "combine_backward", "op": "combine_backward", "W": 8, "tokens": 8192, "E": 64, "k": 2,
         "H": 7168, "dtype": "bf16", "residual": False, "skew": 1.2},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "experts", "experts", "experts_backward",
                     "combine", "combine_backward"])
    W = rng.choice([1, 2, 4, 8])
    tokens = _log_int(rng, 1, 8192)
    if op.startswith("route"):
        grouped = rng.random() < 0.5
        groups = rng.choice([2, 4, 8]) if grouped else 1
        E = groups * _log_int(rng, 4, 256 // groups)
        sigmoid = rng.random() < 0.5
        top_groups = rng.randint(1, groups)
        return {"op": op, "W": W, "tokens": tokens, "E": E,
                "k": rng.randint(1, min(8, top_groups * (E // groups))),
                "dtype": rng.choice(["f32", "bf16", "f16"]),
                "score": "sigmoid" if sigmoid else "softmax", "bias": sigmoid and rng.random() < 0.7,
                "groups": groups, "top_groups": top_groups,
                "group_top": rng.choice([1, 2]) if sigmoid else 1,
                "renormalise": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5])}
    E = W * _log_int(rng, 1, 64 // W)
    k = rng.randint(1, min(4, E))
    skew = rng.choice([0.0, 0.8, 1.2])
    if op.startswith("combine"):
        return {"op": op, "W": W, "tokens": tokens if k <= 2 else (tokens + 1) // 2, "E": E, "k": k,
                "H": _log_int(rng, 65, 7168) if rng.random() < 0.3 else 8 * _log_int(rng, 8, 896),
                "dtype": rng.choice(["bf16", "f16", "f32"]),
                "residual": op == "combine" and rng.random() < 0.5, "skew": skew}
    backward = op == "experts_backward"
    gated = rng.random() < 0.5
    D, N = 8 * _log_int(rng, 16, 896), 8 * _log_int(rng, 16, 896)
    if gated or E > 32:
        N = min(N, 2048)
    rows = (32768 if backward else 131072) * 2048 // max(2048, N)
    return {"op": op, "W": W, "tokens": max(1, min(tokens, rows // (W * k))), "E": E, "k": k,
            "D": D, "N": N,
            "dtype": rng.choice(["bf16", "f16"]),
            "act": rng.choice(["relu", "gelu", "silu"] if gated else ["none", "relu", "gelu", "silu"]),
            "gated": gated, "bias": rng.random() < 0.5,
            "residual": not backward and rng.random() < 0.3, "skew": skew}


# ----------------------------------------------------------------- inputs --
def _popularity(case, device):
    """Experts' popularity: k^-skew, spread over the expert ids by a fixed stride."""
    E = case["E"]
    place = torch.arange(E, device=device, dtype=torch.float32)
    place = (place * 29 + 7) % E if E % 29 else place
    return (place + 1) ** -case["skew"]


def _routing(case, gen):
    """Each rank's choices, [W, T, k] int64: k distinct experts a token, by popularity."""
    W, T, E, k = case["W"], case["tokens"], case["E"], case["k"]
    u = torch.rand((W, T, E), generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)
    score = _popularity(case, "cuda").log() - (-u.log()).log()
    return score.topk(k, dim=-1).indices


def _normal(shape, gen, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _split_rows(flat, rows):
    return list(flat.split(rows))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * int(seed) + 17)
    W, T, E, k, op = case["W"], case["tokens"], case["E"], case["k"], case["op"]
    dt = _DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if op.startswith("route"):
        # logits of a trained router: unit noise around experts that differ
        base = torch.randn(E, generator=gen, device="cuda") * 0.5
        flat = (torch.randn((W * T, E), generator=gen, device="cuda") * 1.5 + base).to(dt)
        s["logits"] = flat
        s["logits_of"] = _split_rows(flat, T)
        s["bias"] = torch.randn(E, generator=gen, device="cuda") * 0.1 if case["bias"] else None
        s["weights"] = torch.empty((W * T, k), device="cuda")
        s["weights_of"] = _split_rows(s["weights"], T)
        s["counts"] = torch.empty((W, E), dtype=torch.int64, device="cuda")
        s["keys"] = torch.empty((W * T, k), dtype=torch.int32, device="cuda")
        s["keys_of"] = _split_rows(s["keys"], T)
        if op == "route_backward":
            s["keys"].copy_(_choose(case, _choice(case, flat, s["bias"])))
            s["d_weights"] = torch.randn((W * T, k), generator=gen, device="cuda")
            s["d_weights_of"] = _split_rows(s["d_weights"], T)
            s["d_logits_of"] = _split_rows(torch.empty_like(flat), T)
        return s
    choices = _routing(case, gen)
    K = E // W
    counts = torch.zeros((W, E), dtype=torch.int64, device="cuda")
    counts.scatter_add_(1, choices.reshape(W, T * k), torch.ones((W, T * k), dtype=torch.int64, device="cuda"))
    rows = counts.view(W, W, K).sum((0, 2)).tolist()  # rows each peer holds
    M = W * T * k
    s["counts"] = counts
    if op.startswith("experts"):
        D, N = case["D"], case["N"]
        Z = 2 * N if case["gated"] else N
        s["rows"] = _normal((M, D), gen, dt)
        s["rows_of"] = _split_rows(s["rows"], rows)
        s["weights"] = torch.empty((E, Z, D), dtype=dt, device="cuda")
        for e in range(E):
            s["weights"][e] = _normal((Z, D), gen, dt, D ** -0.5)
        s["weights_of"] = list(s["weights"].view(W, K, Z, D))
        s["bias"] = _normal((E, Z), gen, dt, 0.2) if case["bias"] else None
        s["bias_of"] = list(s["bias"].view(W, K, Z)) if case["bias"] else None
        if op == "experts":
            s["residual"] = _normal((M, N), gen, dt) if case["residual"] else None
            s["residual_of"] = _split_rows(s["residual"], rows) if case["residual"] else None
            s["out"] = torch.empty((M, N), dtype=dt, device="cuda")
            s["out_of"] = _split_rows(s["out"], rows)
        else:
            s["d_out"] = _normal((M, N), gen, dt)
            s["d_out_of"] = _split_rows(s["d_out"], rows)
            # the pre-activations that the forward pass saved
            plain = case["act"] == "none" and not case["gated"]
            s["pre"] = None if plain else _normal((M, Z), gen, dt)
            s["pre_of"] = None if plain else _split_rows(s["pre"], rows)
            s["d_rows"] = torch.empty((M, D), dtype=dt, device="cuda")
            s["d_rows_of"] = _split_rows(s["d_rows"], rows)
            s["d_weights"] = torch.empty_like(s["weights"])
            s["d_weights_of"] = list(s["d_weights"].view(W, K, Z, D))
            s["d_bias"] = torch.empty_like(s["bias"]) if case["bias"] else None
            s["d_bias_of"] = list(s["d_bias"].view(W, K, Z)) if case["bias"] else None
        return s
    H = case["H"]
    s["in_splits"] = counts.view(W, W, K).sum(2)
    keys = choices.to(torch.int32).reshape(W, T * k)
    order = torch.sort(keys, dim=1, stable=True).indices
    pos = torch.empty_like(order)
    pos.scatter_(1, order, torch.arange(T * k, device="cuda").expand(W, -1).contiguous())
    s["keys"], s["pos"] = keys, pos
    s["keys_of"], s["pos_of"] = list(keys.view(W, T, k)), list(pos)
    s["weights"] = torch.softmax(torch.randn((W * T, k), generator=gen, device="cuda"), -1)
    s["weights_of"] = _split_rows(s["weights"], T)
    s["peers"] = _normal((M, H), gen, dt)
    s["peers_of"] = _split_rows(s["peers"], rows)
    if op == "combine":
        s["residual"] = _normal((W * T, H), gen, dt) if case["residual"] else None
        s["residual_of"] = _split_rows(s["residual"], T) if case["residual"] else None
        s["out_of"] = _split_rows(torch.empty((W * T, H), dtype=dt, device="cuda"), T)
    else:
        s["d_out"] = _normal((W * T, H), gen, dt)
        s["d_out_of"] = _split_rows(s["d_out"], T)
        s["d_peers"] = torch.empty((M, H), dtype=dt, device="cuda")
        s["d_peers_of"] = _split_rows(s["d_peers"], rows)
        s["d_weights_of"] = _split_rows(torch.empty((W * T, k), device="cuda"), T)
    return s


# ------------------------------------------------------------ plain forms --
def _scores(case, x):
    if case["score"] == "softmax":
        e = torch.exp(x - x.amax(-1, keepdim=True))
        return e / e.sum(-1, keepdim=True)
    return 1 / (1 + torch.exp(-x))


def _choice(case, logits, bias):
    """What the experts are chosen by: the order of a softmax is that of its logits."""
    x = logits.float()
    if case["score"] == "softmax" and bias is None and case["group_top"] == 1:
        return x
    c = _scores(case, x)
    return c if bias is None else c + bias


def _choose(case, c):
    c = torch.where(c.isnan(), -math.inf, c)
    G = case["groups"]
    if G > 1:
        per = c.view(c.shape[0], G, -1)
        g = per.sort(dim=-1, descending=True).values[..., :case["group_top"]].sum(-1)
        best = g.sort(dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        keep = torch.zeros_like(g, dtype=torch.bool).scatter_(1, best, True)
        c = torch.where(keep[..., None], per, -math.inf).reshape(c.shape)
    return c.sort(dim=-1, descending=True, stable=True).indices[:, :case["k"]]


def _plain_route(s):
    case = s["case"]
    W, T, E = case["W"], case["tokens"], case["E"]
    p = _scores(case, s["logits"].float())
    ids = _choose(case, _choice(case, s["logits"], s["bias"]))
    w = p.gather(1, ids)
    if case["renormalise"]:
        t = w.sum(-1, keepdim=True)
        w = torch.where(t == 0, 0.0, w / t)
    w = w * case["scale"]
    rank = torch.arange(W, device=ids.device).repeat_interleave(T)[:, None]
    counts = torch.bincount((rank * E + ids).reshape(-1), minlength=W * E).view(W, E)
    return {"keys": _split_rows(ids.to(torch.int32), T), "weights": _split_rows(w, T), "counts": counts}


def _plain_route_backward(s):
    case = s["case"]
    p = _scores(case, s["logits"].float())
    ids = s["keys"].long()
    g = s["d_weights"] * case["scale"]
    sel = p.gather(1, ids)
    if case["renormalise"]:
        t = sel.sum(-1, keepdim=True)
        q = torch.where(t == 0, 0.0, sel / t)
        g = torch.where(t == 0, 0.0, (g - (g * q).sum(-1, keepdim=True)) / t)
    if case["score"] == "sigmoid":
        d = torch.zeros_like(p).scatter_(1, ids, g * sel * (1 - sel))
    elif case["renormalise"]:
        d = torch.zeros_like(p).scatter_(1, ids, g * sel)
    else:
        d = p * (torch.zeros_like(p).scatter_(1, ids, g) - (g * sel).sum(-1, keepdim=True))
    return {"d_logits": _split_rows(d.to(s["logits"].dtype), case["tokens"])}


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


def _act_slope(case, z):
    a = case["act"]
    if a == "relu":
        return (z > 0).to(z.dtype)
    if a == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5
    if a == "silu":
        t = 1 / (1 + torch.exp(-z))
        return t * (1 + z * (1 - t))
    return torch.ones_like(z)


def _rows(x, segments):
    return torch.cat([x[a:b] for a, b in segments]).float()


def _put(out, segments, y):
    at = 0
    for a, b in segments:
        out[a:b] = y[at:at + b - a]
        at += b - a


def _plain_experts(s):
    case = s["case"]
    N = case["N"]
    out = torch.empty((s["rows"].shape[0], N), dtype=s["rows"].dtype, device=s["rows"].device)
    for e, segments in _groups(case, s["counts"]):
        if not segments:
            continue
        z = _rows(s["rows"], segments) @ s["weights"][e].float().T
        if s["bias"] is not None:
            z = z + s["bias"][e].float()
        y = _act(case, z[:, :N]) * z[:, N:] if case["gated"] else _act(case, z)
        if s["residual"] is not None:
            y = y + _rows(s["residual"], segments)
        _put(out, segments, y)
    return {"out": out}


def _plain_experts_backward(s):
    case, N = s["case"], s["case"]["N"]
    d_rows, d_w = torch.empty_like(s["rows"]), torch.zeros_like(s["weights"])
    d_b = None if s["bias"] is None else torch.zeros_like(s["bias"])
    for e, segments in _groups(case, s["counts"]):
        if not segments:
            continue
        dz = _rows(s["d_out"], segments)
        if s["pre"] is not None:
            z = _rows(s["pre"], segments)
            if case["gated"]:
                g, u = z[:, :N], z[:, N:]
                dz = torch.cat([dz * u * _act_slope(case, g), dz * _act(case, g)], 1)
            else:
                dz = dz * _act_slope(case, z)
        _put(d_rows, segments, dz @ s["weights"][e].float())
        d_w[e] = dz.T @ _rows(s["rows"], segments)
        if d_b is not None:
            d_b[e] = dz.sum(0)
    return {"d_rows": d_rows, "d_weights": d_w, "d_bias": d_b}


def _item_rows(s):
    """Row of each item (rank-major) in the peers' rows, all peers one after the other."""
    S, keys, pos = s["in_splits"], s["keys"].long(), s["pos"]
    K = s["case"]["E"] // s["case"]["W"]
    in_off = S.cumsum(1) - S
    sent = S.T.reshape(-1)  # (peer, source)
    out_off = (sent.cumsum(0) - sent).view(S.shape[0], -1)  # [peer][source], over all peers
    peer = keys // K
    return (pos + out_off.T.gather(1, peer) - in_off.gather(1, peer)).reshape(-1)


def _plain_combine(s):
    case = s["case"]
    x = s["peers"][_item_rows(s)].float()
    y = (x.view(-1, case["k"], case["H"]) * s["weights"][..., None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"out": _split_rows(y.to(s["peers"].dtype), case["tokens"])}


def _plain_combine_backward(s):
    case = s["case"]
    at = _item_rows(s)
    dy = s["d_out"].float()[:, None]
    d_w = (s["peers"][at].float().view(-1, case["k"], case["H"]) * dy).sum(-1)
    d = torch.empty_like(s["peers"])
    d[at] = (s["weights"][..., None] * dy).view(-1, case["H"]).to(d.dtype)
    return {"d_peers": d, "d_weights": _split_rows(d_w, case["tokens"])}


_PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward, "experts": _plain_experts,
          "experts_backward": _plain_experts_backward, "combine": _plain_combine,
          "combine_backward": _plain_combine_backward}


# ---------------------------------------------------------- the framework --
def _own_route(s):
    c = s["case"]
    _engine(c["W"]).route(s["logits_of"], s["keys_of"], s["weights_of"], c["k"], counts=s["counts"],
                          bias=s["bias"], score=c["score"], groups=c["groups"],
                          top_groups=c["top_groups"], group_top=c["group_top"],
                          renormalise=c["renormalise"], scale=c["scale"])
    return {"keys": s["keys_of"], "weights": s["weights_of"], "counts": s["counts"]}


def _own_route_backward(s):
    c = s["case"]
    _engine(c["W"]).route_backward(s["logits_of"], s["keys_of"], s["d_weights_of"], s["d_logits_of"],
                                   c["k"], score=c["score"], renormalise=c["renormalise"],
                                   scale=c["scale"])
    return {"d_logits": s["d_logits_of"]}


def _own_experts(s):
    c = s["case"]
    _engine(c["W"]).expert_matmul(s["rows_of"], s["counts"], s["weights_of"], s["out_of"],
                                  activation=c["act"], gated=c["gated"], bias=s["bias_of"],
                                  residual=s["residual_of"])
    return {"out": s["out"]}


def _own_experts_backward(s):
    c = s["case"]
    _engine(c["W"]).expert_matmul_backward(s["rows_of"], s["counts"], s["weights_of"], s["d_out_of"],
                                           d_rows=s["d_rows_of"], d_weights=s["d_weights_of"],
                                           d_bias=s["d_bias_of"], pre=s["pre_of"],
                                           activation=c["act"], gated=c["gated"])
    return {"d_rows": s["d_rows"], "d_weights": s["d_weights"], "d_bias": s["d_bias"]}


def _own_combine(s):
    c = s["case"]
    _engine(c["W"]).combine_weighted(s["peers_of"], s["in_splits"], s["keys_of"], s["pos_of"],
                                     c["E"] // c["W"], s["weights_of"], s["out_of"],
                                     residual=s["residual_of"])
    return {"out": s["out_of"]}


def _own_combine_backward(s):
    c = s["case"]
    _engine(c["W"]).combine_weighted_backward(s["peers_of"], s["in_splits"], s["keys_of"], s["pos_of"],
                                              c["E"] // c["W"], s["weights_of"], s["d_out_of"],
                                              s["d_peers_of"], s["d_weights_of"])
    return {"d_peers": s["d_peers"], "d_weights": s["d_weights_of"]}


_OWN = {"route": _own_route, "route_backward": _own_route_backward, "experts": _own_experts,
        "experts_backward": _own_experts_backward, "combine": _own_combine,
        "combine_backward": _own_combine_backward}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------- work --
def work(case):
    W, T, E, k, op = case["W"], case["tokens"], case["E"], case["k"], case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    tokens, items = W * T, W * T * k
    if op == "route":
        return {"bytes": tokens * E * size + items * 8 + W * E * 8 + (E * 4 if case["bias"] else 0),
                "flops": 4 * tokens * E}
    if op == "route_backward":
        dense = case["score"] == "softmax" and not case["renormalise"]
        return {"bytes": tokens * E * size + (tokens * E if dense else items) * size + items * 8,
                "flops": (8 * tokens * E) if dense else 8 * items}
    if op.startswith("experts"):
        D, N = case["D"], case["N"]
        Z = 2 * N if case["gated"] else N
        pop = _popularity(case, "cpu").double()
        hit = float((1 - (1 - pop / pop.sum()) ** items).sum())  # experts with a row, on average
        flops = 2.0 * items * D * Z
        moved = items * (D + N) * size + hit * Z * D * size
        if op == "experts":
            return {"bytes": moved + (items * N * size if case["residual"] else 0) + W * E * 8,
                    "flops": flops}
        pre = 0 if case["act"] == "none" and not case["gated"] else items * Z * size
        return {"bytes": moved + items * D * size + E * Z * D * size + pre + W * E * 8,
                "flops": 2 * flops}
    H = case["H"]
    if op == "combine":
        return {"bytes": (items + tokens * (2 if case["residual"] else 1)) * H * size + items * 16,
                "flops": 2 * items * H}
    return {"bytes": (2 * items + tokens) * H * size + items * 20, "flops": 3 * items * H}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The definitions in 64 bits.  Choices of experts and counts are whole numbers: none here."""
    s = prepare(case, seed)
    f = {"route": _exact_route, "route_backward": _exact_route_backward, "experts": _exact_experts,
         "experts_backward": _exact_experts, "combine": _exact_combine,
         "combine_backward": _exact_combine}[case["op"]]
    return f(case, s)


def _exact_prob(case, x):
    if case["score"] == "softmax":
        x = x - x.max(axis=1, keepdims=True)
        return np.exp(x) / np.exp(x).sum(axis=1, keepdims=True)
    return 1 / (1 + np.exp(-x))


def _exact_route(case, s):
    W, T, E, k, G = case["W"], case["tokens"], case["E"], case["k"], case["groups"]
    p = _exact_prob(case, s["logits"].double().cpu().numpy())
    c = p if s["bias"] is None else p + s["bias"].double().cpu().numpy()[None]
    if G > 1:
        per = c.reshape(-1, G, E // G)
        score = np.sort(per, axis=2)[:, :, ::-1][:, :, :case["group_top"]].sum(axis=2)
        lost = np.argsort(-score, axis=1, kind="stable")[:, case["top_groups"]:]
        per = per.copy()
        np.put_along_axis(per, lost[:, :, None], -np.inf, axis=1)
        c = per.reshape(-1, E)
    ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, ids, axis=1)
    if case["renormalise"]:
        w = w / w.sum(axis=1, keepdims=True)
    w = w * case["scale"]
    return {"keys": [None] * W, "weights": [w[r * T:(r + 1) * T] for r in range(W)], "counts": None}


def _exact_route_backward(case, s):
    """Through the Jacobian: d logits_i = sum_j g_j d w_j / d x_i."""
    W, T, k = case["W"], case["tokens"], case["k"]
    p = _exact_prob(case, s["logits"].double().cpu().numpy())
    ids = s["keys"].cpu().numpy().astype(np.int64)
    g = s["d_weights"].double().cpu().numpy() * case["scale"]
    sel = np.take_along_axis(p, ids, axis=1)
    if case["renormalise"]:
        t = sel.sum(axis=1, keepdims=True)
        g = g / t - (g * sel).sum(axis=1, keepdims=True) / (t * t)
    onto = np.zeros_like(p)
    np.put_along_axis(onto, ids, g, axis=1)  # the gradient with respect to the scores
    d = onto * p * (1 - p) if case["score"] == "sigmoid" else \
        p * onto - p * (p * onto).sum(axis=1, keepdims=True)
    return {"d_logits": [d[r * T:(r + 1) * T] for r in range(W)]}


def _exact_experts(case, s):
    W, K, N = case["W"], case["E"] // case["W"], case["N"]
    counts = s["counts"].cpu().numpy()
    backward = case["op"] == "experts_backward"
    results = {"out": []} if not backward else {"d_rows": [], "d_weights": [], "d_bias": []}
    half = 0.5 ** 0.5

    def phi(z):  # the standard normal's distribution function
        return 0.5 * torch.erfc(-z * half)

    def act(z):
        return {"none": lambda: z, "relu": lambda: torch.relu(z), "gelu": lambda: z * phi(z),
                "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()

    def slope(z):
        if case["act"] == "none":
            return torch.ones_like(z)
        if case["act"] == "relu":
            return torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
        if case["act"] == "gelu":
            return phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)

    for p in range(W):
        n = s["rows_of"][p].shape[0]
        # the expert of each row of this peer: (source, local expert) in order
        owner = torch.from_numpy(np.tile(np.arange(K), W).repeat(counts[:, p * K:(p + 1) * K].reshape(-1))).cuda()
        x, w = s["rows_of"][p], s["weights_of"][p]
        out = torch.zeros((n, x.shape[1] if backward else N), dtype=torch.float64, device="cuda")
        d_w = torch.zeros(w.shape, dtype=torch.float64, device="cuda") if backward else None
        d_b = torch.zeros(w.shape[:2], dtype=torch.float64, device="cuda")
        for e in range(K):
            at = (owner == e).nonzero().reshape(-1)
            xe, we = x[at].double(), w[e].double()
            if not backward:
                z = torch.einsum("md,nd->mn", xe, we)
                if s["bias"] is not None:
                    z += s["bias_of"][p][e].double()
                y = act(z[:, :N]) * z[:, N:] if case["gated"] else act(z)
                if s["residual"] is not None:
                    y += s["residual_of"][p][at].double()
                out[at] = y
                continue
            dz = s["d_out_of"][p][at].double()
            if case["gated"]:
                z = s["pre_of"][p][at].double()
                dz = torch.cat([dz * z[:, N:] * slope(z[:, :N]), dz * act(z[:, :N])], dim=1)
            elif case["act"] != "none":
                dz = dz * slope(s["pre_of"][p][at].double())
            out[at] = torch.einsum("mn,nd->md", dz, we)
            d_w[e] = torch.einsum("mn,md->nd", dz, xe)
            d_b[e] = dz.sum(0)
        results["d_rows" if backward else "out"].append(out)
        if backward:
            results["d_weights"].append(d_w)
            results["d_bias"].append(d_b)
    results = {name: torch.cat(v) for name, v in results.items()}
    if backward:
        results["d_weights"] = results["d_weights"].view(s["weights"].shape)
        results["d_bias"] = results["d_bias"].view(s["bias"].shape) if s["bias"] is not None else None
    return results


def _exact_combine(case, s):
    W, T, k, K = case["W"], case["tokens"], case["k"], case["E"] // case["W"]
    S = s["in_splits"].cpu().numpy()
    keys, pos = s["keys"].cpu().numpy(), s["pos"].cpu().numpy()
    backward = case["op"] == "combine_backward"
    d_peers = [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in s["peers_of"]] if backward else None
    ys, dws = [], []
    for r in range(W):
        w = s["weights_of"][r].double()
        y = torch.zeros((T, case["H"]), dtype=torch.float64, device="cuda")
        d_w = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        if not backward and s["residual"] is not None:
            y += s["residual_of"][r].double()
        for p in range(W):
            item = np.nonzero(keys[r] // K == p)[0]
            row = torch.from_numpy(S[:r, p].sum() + pos[r][item] - S[r, :p].sum()).cuda()
            t, j = torch.from_numpy(item // k).cuda(), torch.from_numpy(item % k).cuda()
            x = s["peers_of"][p][row].double()
            if backward:
                dy = s["d_out_of"][r][t].double()
                d_peers[p][row] = w[t, j][:, None] * dy
                d_w[t, j] = (x * dy).sum(1)
            else:
                y.index_add_(0, t, w[t, j][:, None] * x)
        ys.append(y)
        dws.append(d_w)
    return {"d_peers": torch.cat(d_peers), "d_weights": dws} if backward else {"out": ys}
