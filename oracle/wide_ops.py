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


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row's token, from the definition: float64 weights, the order of falling logits
    (equal ones by number). Also returns how near u and top-p came to another answer, as a
    part of the sums that they divide."""
    x = np.array(logits, dtype=np.float64)
    x[np.isnan(x)] = -np.inf
    top = x.max()
    if top == -np.inf:
        return -1, 1.0
    if temperature == 0 or top_k == 1 or top_p <= 0 or min_p > 1:
        return int(np.argmax(x)), 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / temperature))
    order = np.lexsort((np.arange(len(x)), -x))
    kept = order[:top_k] if 0 < top_k < len(x) else order
    near = 1.0
    if top_p < 1:
        upto = np.cumsum(w[kept])
        target = top_p * upto[-1]
        before = np.concatenate([[0.0], upto[:-1]])
        near = np.abs(upto[upto < upto[-1]] - target).min(initial=np.inf) / upto[-1]
        kept = kept[(before < target) | (np.arange(len(kept)) == 0)]
    kept = np.sort(kept[w[kept] >= min_p])
    upto = np.cumsum(w[kept])
    target = u * upto[-1]
    inner = upto[:-1]
    if u < 1:  # 1 is the last one with a weight, however small
        near = min(near, np.abs(inner - target).min(initial=np.inf) / upto[-1])
    i = int(np.searchsorted(upto, target, side="right"))
    if i >= len(kept):  # u = 1: the last one with a weight
        i = int(np.max(np.nonzero(w[kept])[0]))
    return int(kept[i]), float(near)
