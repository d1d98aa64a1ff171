"""Packed rows and the norm from their definitions, in 64 bits with numpy: what
the GPU tests compare the kernels with."""
from __future__ import annotations

import numpy as np

BLOCK = 32
MOST = {"mxfp8": 448.0, "mxfp4": 6.0}
# half a step of a code, relative to the value and, near 0, to the scale
HALF = {"mxfp8": (2.0 ** -4, 2.0 ** -10), "mxfp4": (2.0 ** -2, 2.0 ** -2)}


def _table(fmt):
    """The values of the codes without sign, ascending: 0 .. 126 or 0 .. 7."""
    if fmt == "mxfp4":
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    return np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                     for e in range(16) for m in range(8)][:127])


TABLE = {fmt: _table(fmt) for fmt in MOST}


def layout(D, fmt):
    """Bytes of the values, of the scales and of the row."""
    blocks = -(-D // BLOCK)
    values = blocks * (32 if fmt == "mxfp8" else 16)
    return values, blocks, -(-(values + blocks) // 32) * 32


def scales_of(x, fmt):
    """Scale bytes of blocks [..., 32], one at a time, by trying powers of two."""
    out = np.zeros(x.shape[:-1], np.int64)
    for i in np.ndindex(out.shape):
        top = np.abs(x[i]).max()
        if not np.isfinite(top):
            out[i] = 255
            continue
        s = 0
        if top > 0:
            s = max(0, int(np.floor(np.log2(top))) + 127 - 10)
        while top > MOST[fmt] * 2.0 ** (s - 127):
            s += 1
        out[i] = s
    return out


def codes_of(v, fmt):
    """The nearest codes, ties to the even one, with their sign."""
    t = TABLE[fmt]
    a = np.minimum(np.abs(v), t[-1])
    hi = np.minimum(np.searchsorted(t, a), len(t) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = t[hi] - a, a - t[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code + np.signbit(v) * len(t if fmt == "mxfp4" else range(128))).astype(np.uint8)


def blocks_of(x):
    D = x.shape[1]
    pad = -D % BLOCK
    return np.concatenate([x, np.zeros((x.shape[0], pad))], 1).reshape(x.shape[0], (D + pad) // BLOCK, BLOCK)


def pack(x, fmt):
    """Packed rows of [rows, D] 64-bit values."""
    rows, D = x.shape
    b = blocks_of(x)
    s = scales_of(b, fmt)
    bad = s == 255
    with np.errstate(invalid="ignore"):
        v = np.where(bad[..., None], 0.0, b / 2.0 ** (np.where(bad, 127, s)[..., None] - 127.0))
    c = codes_of(v, fmt).reshape(rows, v.shape[1] * BLOCK)
    if fmt == "mxfp4":
        c = c[:, 0::2] | c[:, 1::2] << 4
    out = np.zeros((rows, layout(D, fmt)[2]), np.uint8)
    out[:, :c.shape[1]] = c
    out[:, c.shape[1]:c.shape[1] + s.shape[1]] = s
    return out


def unpack(rows, D, fmt):
    """(values, the scale of each) of packed rows."""
    V, B, _ = layout(D, fmt)
    c = rows[:, :V]
    if fmt == "mxfp4":
        c = np.stack([c & 15, c >> 4], -1).reshape(rows.shape[0], 2 * V)
        t = np.concatenate([TABLE[fmt], -TABLE[fmt]])
    else:
        t = np.concatenate([TABLE[fmt], [np.nan], -TABLE[fmt], [np.nan]])
    s = rows[:, V:V + B].astype(np.int64)
    scale = np.where(s == 255, np.nan, 2.0 ** (s - 127.0)).repeat(BLOCK, 1)
    return (t[c] * scale)[:, :D], scale[:, :D]


def norm(s, w, eps):
    with np.errstate(all="ignore"):
        return s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * w


def norm_backward(s, w, dy, eps):
    """(d_s, the terms of d_weight, magnitudes of d_s's terms)."""
    r = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    g = dy * w
    mean = (g * s).mean(-1, keepdims=True)
    size = r * np.abs(g) + np.abs(s) * r ** 3 * np.abs(g * s).mean(-1, keepdims=True)
    return r * g - s * r ** 3 * mean, dy * s * r, size


def norm_error(H):
    """Relative error of a row's scale in 32 bits: H squares summed in any order, the
    mean, eps, the root, and the two products after it."""
    return (H / 2 + 8) * 2.0 ** -24
