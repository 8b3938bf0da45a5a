"""The paged key/value cache's operators by their definitions, in 64 bits:
a step's plan, the norm and the rotary embedding of heads, attention row by
row, and pages released, forked and compacted.  Plain numpy and Python; shares
nothing with the GPU path."""
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


def norm(x, weight, eps):
    """x (tokens, heads, dim) float64: every head over the root of its mean
    square, times weight (dim)."""
    x = np.array(x, np.float64)
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            square = sum(float(v) * float(v) for v in x[t, h]) / x.shape[2]
            x[t, h] = x[t, h] * np.asarray(weight, np.float64) / np.sqrt(square + eps)
    return x


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


def attention(q, k, v, scale, causal=True, window=0, sinks=0):
    """One request: q (n, heads, dim), k and v (s, kv_heads, dim), float64; a
    row sees its window and the first `sinks` tokens.  Returns out, lse (n, heads), and per row what error bounds need: the
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
        seen = [j for j in range(hi) if j >= lo or j < sinks]
        if not seen:
            continue
        for h in range(heads):
            g = h // (heads // kv_heads)
            z = scale * (k[seen, g] @ q[i, h])
            m = z.max()
            e = np.exp(z - m)
            w = e / e.sum()
            out[i, h] = w @ v[seen, g]
            spread[i, h] = w @ np.abs(v[seen, g])
            lse[i, h] = m + np.log(e.sum())
            top[i, h] = np.abs(z).max()
            mass[i, h] = scale * (np.abs(k[seen, g]) @ np.abs(q[i, h])).max()
    return out, lse, spread, top, mass


def release(held, keep, table, ring, cursor, shared, page_size, window=0, sinks=0):
    """(table, ring, cursor, shared, cut) after requests are cut to `keep`
    tokens; cut: those cut inside a page that others hold afterwards."""
    table, ring, shared = (np.array(x, np.int32) for x in (table, ring, shared))
    head, tail = (int(x) for x in cursor)
    left = {p: int(s) + 1 for p, s in enumerate(shared)}
    for r, (h, k) in enumerate(zip(map(int, held), map(int, keep))):
        for i in range(-(-h // page_size)):
            tokens = range(i * page_size, (i + 1) * page_size)
            behind = tokens[0] >= k
            passed = window > 0 and all(sinks <= j <= k - window for j in (tokens[0], tokens[-1]))
            if (behind or passed) and table[r, i] >= 0:
                left[int(table[r, i])] -= 1
                table[r, i] = -1
    for p in sorted(left):
        if left[p] == 0:
            ring[tail % len(ring)] = p
            tail += 1
        shared[p] = max(left[p] - 1, 0)
    cut = [r for r, (h, k) in enumerate(zip(map(int, held), map(int, keep)))
           if 0 < k < h and k % page_size and table[r, k // page_size] >= 0 and shared[table[r, k // page_size]] > 0]
    return table, ring, np.array([head, tail], np.int64), shared, cut


def fork(context, parents, table, ring, cursor, shared, page_size, lens=None):
    """(context, table, shared, cursor, src, dst) after requests became copies
    of others.  Sound inputs and a ring with room only."""
    table, shared, context = (np.array(x, np.int32) for x in (table, shared, context))
    head, tail = (int(x) for x in cursor)
    src, dst = [], []
    for r, p in enumerate(map(int, parents)):
        src.append(-1)
        dst.append(-1)
        if p < 0:
            continue
        n = int(context[p]) if lens is None else int(lens[r])
        for i in range(n // page_size):
            table[r, i] = table[p, i]
            if table[p, i] >= 0:
                shared[table[p, i]] += 1
        if n % page_size:
            src[r], dst[r] = int(table[p, n // page_size]), int(ring[head % len(ring)])
            table[r, n // page_size] = dst[r]
            head += 1
        context[r] = n
    return context, table, shared, np.array([head, tail], np.int64), np.array(src, np.int32), np.array(dst, np.int32)


def compact(context, table, ring, cursor, shared, page_size):
    """(table, ring, shared, src, dst) with the held pages the lowest."""
    table, ring, shared = (np.array(x, np.int32) for x in (table, ring, shared))
    head, tail = (int(x) for x in cursor)
    rows = [(r, i) for r, c in enumerate(context) for i in range(-(-int(c) // page_size)) if table[r, i] >= 0]
    held = {int(table[r, i]) for r, i in rows}
    free = {int(ring[k % len(ring)]) for k in range(head, tail)}
    order = sorted(held | free)
    low = set(order[: len(held)])
    src, dst = sorted(held - low), sorted(free & low)
    to = dict(zip(src, dst))
    for r, i in rows:
        table[r, i] = to.get(int(table[r, i]), int(table[r, i]))
    for a, b in to.items():
        shared[b], shared[a] = shared[a], 0
    for k, p in enumerate(order[len(held):]):
        ring[(head + k) % len(ring)] = p
    pad = [-1] * (len(shared) // 2 - len(src))
    return table, ring, shared, np.array(src + pad, np.int32), np.array(dst + pad, np.int32)
