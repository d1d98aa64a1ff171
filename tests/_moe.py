"""The MoE operators from their definitions, in 64 bits with numpy, one token
or one expert at a time: what the GPU tests compare the kernels with."""
from __future__ import annotations

import math

import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# largest relative error of a rounding to the type: 2^-p for p significant bits
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}


# ----------------------------------------------------------------- routing --
def scores(x, score):
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-x))
        m = x.max()
        if m == -np.inf:
            return np.zeros_like(x)
        e = np.exp(x - m)
        return e / e.sum()


def choose(c, k, groups, top_groups, group_top):
    """Experts of the k largest of a token's choices c; ties go to the lowest index."""
    c = np.where(np.isnan(c), -np.inf, c)
    if groups > 1:
        per = c.reshape(groups, -1)
        g = np.array([np.sort(row)[::-1][:group_top].sum() for row in per], dtype=c.dtype)
        keep = np.argsort(-g, kind="stable")[:top_groups]
        lost = np.setdiff1d(np.arange(groups), keep)
        per = per.copy()
        per[lost] = -np.inf
        c = per.reshape(-1)
    return np.argsort(-c, kind="stable")[:k]


def weights_of(x, ids, score, renormalise, scale):
    s = scores(x, score)[ids]
    if renormalise:
        if score == "softmax":
            s = scores(x[ids], score)
        t = s.sum()
        s = s * 0 if t == 0 else s / t
    return s * scale


def weights_gradient(x, ids, g, score, renormalise, scale):
    """d (sum_j g_j w_j) / d x."""
    d = np.zeros_like(x)
    g = g * scale
    s = scores(x, score)
    if score == "softmax" and not renormalise:
        gi = np.zeros_like(x)
        gi[ids] = g
        return s * (gi - (gi * s).sum())
    if score == "softmax":
        q = scores(x[ids], score)
        d[ids] = q * (g - (g * q).sum())
        return d
    sj = s[ids]
    if renormalise:
        t = sj.sum()
        if t == 0:
            return d
        g = (g - (g * sj).sum() / t) / t
    d[ids] = g * sj * (1 - sj)
    return d


# ----------------------------------------------------------------- experts --
_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(name, z):
    if name == "relu":
        return np.where(z < 0, 0, z)
    if name == "gelu":
        return z * 0.5 * (1 + _erf(z / math.sqrt(2)))
    if name == "silu":
        return z / (1 + np.exp(-z))
    return z


def slope(name, z):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def row_experts(counts, p, K):
    """The local expert of each of peer p's rows: (source rank, expert) in order."""
    W = counts.shape[0]
    return np.concatenate([np.repeat(np.arange(K), counts[r, p * K:(p + 1) * K]) for r in range(W)])


def f64(t):
    return t.detach().double().cpu().numpy()


def expert_forward(x, owner, w, b, res, name, gated):
    """One peer: (y, z, bound), bound on a 32-bit sum's error carried to y."""
    C, K = x.shape[1], w.shape[0]
    N = w.shape[1] // 2 if gated else w.shape[1]
    z = np.zeros((x.shape[0], w.shape[1]))
    mag = np.zeros_like(z)
    for e in range(K):
        at = owner == e
        z[at] = x[at] @ w[e].T + (0 if b is None else b[e])
        mag[at] = np.abs(x[at]) @ np.abs(w[e]).T + (0 if b is None else np.abs(b[e]))
    dz = (C + 8) * 2.0 ** -24 * mag  # any order of a sum of C products and the bias
    if gated:
        g, u = z[:, :N], z[:, N:]
        y = act(name, g) * u
        # the activations' slopes are below 1.13; the fast exponential's and
        # divide's own errors stay below 2^-18 of the result
        bound = 1.13 * dz[:, :N] * (np.abs(u) + dz[:, N:]) + np.abs(act(name, g)) * dz[:, N:]
    else:
        y, bound = act(name, z), 1.13 * dz
    # the error function's tail: 1 + erf loses its relative precision below 0
    bound = bound + 2.0 ** -18 * np.abs(y) + (2.0 ** -22 * np.abs(z).max(initial=0) if name == "gelu" else 0)
    if gated and name == "gelu":
        bound = bound + 2.0 ** -22 * np.abs(z).max(initial=0) * np.abs(z[:, N:])
    if res is not None:
        y = y + res
    return y, z, bound, dz


def expert_dz(dy, pre, name, gated):
    if not gated:
        return dy * slope(name, pre) if name != "none" else dy
    N = dy.shape[1]
    g, u = pre[:, :N], pre[:, N:]
    return np.concatenate([dy * u * slope(name, g), dy * act(name, g)], axis=1)


def close(got, ref, bound, dtype, what):
    """|got - ref| <= the rounding to the type + `bound`, element by element."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    limit = UNIT[dtype] * (np.abs(ref) + bound) * 1.01 + TINY[dtype] + bound
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - ref) <= limit) & ~(np.isnan(got) & np.isnan(ref))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} values differ, first at {i}: "
                             f"{got[i]} against {ref[i]}, limit {limit[i]}")
