"""Float64 CPU statements of the operators between the int4 projections.

Plain numpy and Python loops from the formulas, for the tests only. Inputs are
float64 arrays holding the exact values of the GPU tensors; results come with the
magnitudes that error bounds are made of (sums of absolute values in the place of
sums).
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def kv_extend(lens, new_tokens, table, free_pages, free_count, page_size, n_slots, spacing=0):
    """The step's places, one request and one token after the other. Returns a dict
    with the names of the call's outputs (table and free_pages as they are left)."""
    lens, new = [int(x) for x in lens], [int(x) for x in new_tokens]
    table, free = np.array(table), np.array(free_pages)
    max_pages, pool = table.shape[1], len(free)
    pages = lambda n: -(-n // page_size)  # noqa: E731
    room = min(max_pages * page_size, 2**31 - 1)
    stack = [int(x) for x in free[:min(max(int(free_count), 0), pool)]]
    given = []
    for b, n in enumerate(new):
        if n < 0:
            given += [int(x) for x in table[b, :min(pages(max(lens[b], 0)), max_pages)]]
    for x in given:
        if len(stack) < pool:
            free[len(stack)] = x
            stack.append(x)
    count, total_need, taken, at = len(stack), 0, 0, 0
    lens_out, refused = list(lens), [0] * len(lens)
    slots, positions = np.full(n_slots, -1, dtype=np.int64), np.zeros(n_slots, dtype=np.int32)
    for b, n in enumerate(new):
        if n < 0:
            lens_out[b] = 0
            continue
        start = b * spacing if spacing else at
        at = start + n
        if lens[b] < 0 or lens[b] + n > room or (n > 0 and (at > n_slots or (spacing and n > spacing))):
            refused[b] = 2
            continue
        held, need = pages(lens[b]), pages(lens[b] + n) - pages(lens[b])
        total_need += need
        if need and total_need > count:
            refused[b] = 1
            continue
        for i in range(need):
            table[b, held + i] = stack[count - 1 - (total_need - need + i)]
        if need:
            taken = total_need
        lens_out[b] = lens[b] + n
        for i in range(n):
            pos = lens[b] + i
            positions[start + i] = pos
            page = int(table[b, pos // page_size])
            slots[start + i] = page * page_size + pos % page_size if page >= 0 else -1
    return {"table": table, "free_pages": free, "free_count_out": count - taken, "lens_out": np.array(lens_out),
            "refused": np.array(refused), "slots": slots, "positions": positions}


def rope(x, positions, inv_freq, rot_dim, interleaved, mscale):
    """x [rows, heads, D] turned; returns (turned, magnitude)."""
    x = np.asarray(x, dtype=np.float64)
    two_pi = np.longdouble(2) * np.arctan2(np.longdouble(0), np.longdouble(-1))
    angle = np.asarray(positions).astype(np.longdouble)[:, None] * np.asarray(inv_freq).astype(np.longdouble)[None, :]
    angle = np.mod(angle, two_pi).astype(np.float64)[:, None, :]
    c, s = mscale * np.cos(angle), mscale * np.sin(angle)
    i = np.arange(rot_dim // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)
    out, mag = x.copy(), np.abs(x)
    out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
    out[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    mag[:, :, a] = mag[:, :, b] = abs(mscale) * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
    return out, mag


def attention(q, k, v, scale, softcap=0.0):
    """One request and kv head: q [group, D] over k, v [tokens, D]. Returns out [group, D],
    lse [group], the mean of |v| under the weights [group, D] and the largest
    scale * sum |q k| [group]."""
    g, D = q.shape
    if len(k) == 0:
        return np.zeros((g, D)), np.full(g, -np.inf), np.zeros((g, D)), np.zeros(g)
    s = scale * (q @ k.T)
    if softcap:
        s = softcap * np.tanh(s / softcap)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(axis=1, keepdims=True)
    return ((p @ v) / total, (m + np.log(total))[:, 0], (p @ np.abs(v)) / total,
            (abs(scale) * (np.abs(q) @ np.abs(k).T)).max(axis=1))


def residual_rmsnorm(h, y, gamma, eps, post_gamma=None, gate=None, alpha=1.0):
    """Returns (h_out, n_out, magnitude of h_out, magnitude of n_out)."""
    rms = lambda x: np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)  # noqa: E731
    t = np.asarray(y, dtype=np.float64)
    if post_gamma is not None:
        t = t / rms(t) * post_gamma
    if gate is not None:
        t = t * gate
    out = h + alpha * t
    mag = np.abs(h) + np.abs(alpha * t)
    n = None if gamma is None else out / rms(out) * gamma
    return out, n, mag, None if gamma is None else mag / rms(out) * np.abs(gamma)
