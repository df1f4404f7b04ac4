"""8-bit blocks and the products over them on the CPU.

A value is an e4m3 code times the scale of its block of 128: s = max(max |y| / 448,
2^-126), q = e4m3(y / s), both quotients rounded to float32 first, ties to even; a
NaN or an infinity makes the block's scale and codes NaN.  Rows have a scale for
each 128 columns, [column block, row]; weights one for each 128 x 128 block.

Values are float64 unless a rounding is named; nothing is shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from oracle.kv4 import E4M3, nearest

B = 128
TINY = 2.0 ** -126


def blocks(n):
    return -(-n // B)


def code_values(x):
    """The e4m3 values nearest to x (NaN stays), saturating at 448."""
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    return np.where(np.isnan(x), np.nan, np.copysign(E4M3[nearest(np.minimum(a, 448.0), E4M3)], x))


def block_scale(y):
    """The scale of one block of values, a float32 held in float64."""
    top = np.abs(y).max(initial=0.0) if np.isfinite(y).all() else np.nan
    return np.float64(np.maximum(np.float32(top) / np.float32(448), np.float32(TINY))) if np.isfinite(top) else np.nan


def _quantised(y, s):
    with np.errstate(invalid="ignore"):
        return code_values((y.astype(np.float32) / np.float32(s)).astype(np.float64)) if np.isfinite(s) else np.full(y.shape, np.nan)


def quantise_rows(y):
    """float32 values [rows, n] -> (code values [rows, n], scales [ceil(n / 128), rows])."""
    q, s = np.empty(y.shape), np.empty((blocks(y.shape[1]), y.shape[0]))
    for r in range(y.shape[0]):
        for b in range(s.shape[0]):
            part = y[r, b * B:(b + 1) * B]
            s[b, r] = block_scale(part)
            q[r, b * B:(b + 1) * B] = _quantised(part, s[b, r])
    return q, s


def quantise_weights(w):
    """float32 values [rows, n] -> (code values, scales [ceil(rows / 128), ceil(n / 128)])."""
    q, s = np.empty(w.shape), np.empty((blocks(w.shape[0]), blocks(w.shape[1])))
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = (slice(i * B, (i + 1) * B), slice(j * B, (j + 1) * B))
            s[i, j] = block_scale(w[at])
            q[at] = _quantised(w[at], s[i, j])
    return q, s


def rows_of(q, s):
    """The values that 8-bit rows stand for."""
    return q * np.repeat(s.T, B, 1)[:, :q.shape[1]]


def weights_of(q, s):
    """The values that an 8-bit weight matrix stands for."""
    return q * np.repeat(np.repeat(s, B, 0)[:q.shape[0]], B, 1)[:, :q.shape[1]]


def norm(x, r, g, eps):
    """(h, y): h = x + r, y = h g / sqrt(mean(h^2) + eps)."""
    h = x if r is None else x + r
    return h, h * g / np.sqrt((h * h).mean(-1, keepdims=True) + eps)


def swiglu(gate, up):
    with np.errstate(over="ignore"):
        return gate / (1 + np.exp(-gate)) * up
