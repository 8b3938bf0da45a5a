"""The paged key/value cache's operators by their definitions, in 64 bits:
a step's plan, the rotary embedding, and attention row by row.  Plain numpy
and Python; shares nothing with the GPU path."""
from __future__ import annotations

import numpy as np


def plan(context, new, table, free, cursor, page_size, tokens):
    """(table, seq_lens, cu_q, slots, positions, cursor) after a step."""
    table = [list(map(int, row)) for row in np.asarray(table)]
    head, tail = (int(x) for x in cursor)
    at = head
    slots, positions, cu, lens = [], [], [0], []
    for r, (c, n) in enumerate(zip(map(int, context), map(int, new))):
        for i in range(-(-c // page_size), -(-(c + n) // page_size)):
            table[r][i] = int(free[at % len(free)]) if at < tail else -1
            at += 1
        for pos in range(c, c + n):
            page = table[r][pos // page_size]
            slots.append(page * page_size + pos % page_size if page >= 0 else -1)
            positions.append(pos)
        lens.append(c + n)
        cu.append(cu[-1] + n)
    pad = tokens - len(slots)
    return (np.array(table, np.int32), np.array(lens, np.int32), np.array(cu, np.int32),
            np.array(slots + [-1] * pad, np.int64), np.array(positions + [0] * pad, np.int32),
            np.array([min(at, tail), tail], np.int64))


def rotate(x, positions, table, interleaved):
    """x (tokens, heads, dim) float64, table (positions, rot) cosines | sines."""
    x = np.array(x, np.float64)
    half = table.shape[1] // 2
    for t, p in enumerate(positions):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = float(table[p, i]), float(table[p, half + i])
            u, w = x[t, :, a].copy(), x[t, :, b].copy()
            x[t, :, a] = u * c - w * s
            x[t, :, b] = w * c + u * s
    return x


def gather(cache, table, page_size, n):
    """The first n tokens' rows (n, kv_heads, dim) of a request from its pages."""
    return np.stack([cache[table[j // page_size], j % page_size] for j in range(n)]) if n else \
        np.zeros((0,) + cache.shape[2:], cache.dtype)


def attention(q, k, v, scale, causal=True, window=0):
    """One request: q (n, heads, dim), k and v (s, kv_heads, dim), float64.
    Returns out, lse (n, heads), and per row what error bounds need: the
    weighted sum of |v| (n, heads, dim), the largest |scaled score| and the
    largest sum of |scale q_i k_i| over its keys (n, heads)."""
    n, heads, dim = q.shape
    s, kv_heads, _ = k.shape
    out = np.zeros(q.shape)
    spread = np.zeros(q.shape)
    lse = np.full((n, heads), -np.inf)
    top = np.zeros((n, heads))
    mass = np.zeros((n, heads))
    for i in range(n):
        p = s - n + i
        lo = max(0, p - window + 1) if window else 0
        hi = min(s, p + 1) if causal else s
        if hi <= lo:
            continue
        for h in range(heads):
            g = h // (heads // kv_heads)
            z = scale * (k[lo:hi, g] @ q[i, h])
            m = z.max()
            e = np.exp(z - m)
            w = e / e.sum()
            out[i, h] = w @ v[lo:hi, g]
            spread[i, h] = w @ np.abs(v[lo:hi, g])
            lse[i, h] = m + np.log(e.sum())
            top[i, h] = np.abs(z).max()
            mass[i, h] = scale * (np.abs(k[lo:hi, g]) @ np.abs(q[i, h])).max()
    return out, lse, spread, top, mass
