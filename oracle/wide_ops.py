"""Float64 CPU statements of attention with several new tokens a request and with shared
prefixes, and of the choice of the next token. For the tests only.
"""
from __future__ import annotations

import numpy as np

from .decode_ops import attention


def rows_attention(q, keys, values, position, scale, window=0, softcap=0.0):
    """One request: q [n, heads, D], the last n of the tokens that keys and values
    [tokens, kv_heads, D] hold; row i is at `position` + i and sees the tokens up to there.
    Returns out, lse, the mean of |v| under the weights and the largest scale * sum |q k|,
    each [n, heads, ...]."""
    n, heads, D = q.shape
    kv = keys.shape[1]
    group = heads // kv
    out, mag = np.zeros((n, heads, D)), np.zeros((n, heads, D))
    lse, top = np.full((n, heads), -np.inf), np.zeros((n, heads))
    for i in range(n):
        hi = max(0, min(len(keys), position + i + 1))
        lo = max(0, hi - window) if window else 0
        for j in range(kv):
            at = slice(j * group, (j + 1) * group)
            out[i, at], lse[i, at], mag[i, at], top[i, at] = attention(q[i, at], keys[lo:hi, j], values[lo:hi, j], scale,
                                                                      softcap)
    return out, lse, mag, top
