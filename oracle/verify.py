"""Verification of drafted tokens by its definition, in 64 bits: which drafts
hold against the model's probabilities, and the token that follows them, from
given random numbers.  Plain numpy and Python; shares nothing with the GPU
path."""
from __future__ import annotations

import math

import numpy as np


def softmax(z, temperature):
    """Probabilities of a row of logits (float64); a temperature of 0: one at
    the first of the largest.  None where there are none."""
    z = np.asarray(z, np.float64)
    if not (0 <= temperature < math.inf) or not (z < math.inf).all() or not (z > -math.inf).any():
        return None
    if temperature == 0:
        p = np.zeros(len(z))
        p[int(np.flatnonzero(z == z.max())[0])] = 1.0
        return p
    e = np.exp((z - z.max()) / temperature)
    return e / math.fsum(e)


def pick(weights, u):
    """The first index whose prefix sum is above u times the whole, and how far
    the nearest prefix sum is from it, as a share of the whole."""
    u = 0.0 if not u >= 0 else min(u, 1 - 2.0 ** -24)
    sums = np.cumsum(np.asarray(weights, np.longdouble))
    share = u * sums[-1]
    j = int(np.flatnonzero((sums > share) & (np.asarray(weights) > 0))[0])
    return j, float(np.abs(sums - share).min() / sums[-1])


def request(logits, drafts, uniforms, draft_logits=None, temperature=1.0):
    """One request: logits (n, V), drafts and uniforms (n).  Returns accepted,
    token, and the least distance of any comparison from its border (relative),
    below which roundings decide."""
    n = len(logits)
    margin = math.inf
    for i in range(n):
        p = softmax(logits[i], temperature)
        if p is None:
            return i, -1, margin
        if i == n - 1:
            w = p
            break
        x = int(drafts[i])
        there = 0 <= x < len(p)
        q = np.zeros(len(p))
        if there:
            q[x] = 1.0
        if draft_logits is not None and temperature > 0:
            q = softmax(draft_logits[i], temperature)
            if q is None:
                return i, -1, margin
        px, qx = (p[x], q[x]) if there else (0.0, 1.0)
        u = float(uniforms[i])
        bar = (u if u != u else min(max(u, 0.0), 1 - 2.0 ** -24)) * qx
        if px > 0 and temperature > 0:
            margin = min(margin, abs(bar - px) / px)
        if not bar < px:
            w = np.maximum(p - q, 0)
            if not w.sum() > 0:
                w = p
            break
    token, near = pick(w, float(uniforms[n - 1]))
    if temperature > 0:
        margin = min(margin, near)
    return i, token, margin
