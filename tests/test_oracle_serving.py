"""The serving operators' oracle (oracle/paged.py, oracle/verify.py) on
hand-worked cases and against second forms."""
import math

import numpy as np
import pytest

from oracle import paged as op
from oracle import verify as ov


def test_norm_by_hand():
    x = np.array([[[3.0, 4.0], [0.0, 0.0]]])
    got = op.norm(x, [2.0, 1.0], 0.5)
    root = math.sqrt((9 + 16) / 2 + 0.5)
    assert np.allclose(got, [[[6 / root, 4 / root], [0, 0]]], rtol=1e-15)


def test_sinks_by_hand_and_against_a_mask():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((11, 2, 8)), rng.standard_normal((11, 2, 8))
    for window, sinks in ((1, 1), (3, 2), (4, 20), (3, 0), (0, 5)):
        out, lse, *_ = op.attention(q, k, v, 0.5, window=window, sinks=sinks)
        p, j = np.arange(6, 11)[:, None], np.arange(11)[None, :]
        seen = (j <= p) & ((j > p - window) | (j < sinks) if window else True)
        for h in range(4):
            z = np.where(seen, 0.5 * q[:, h] @ k[:, h // 2].T, -np.inf)
            e = np.exp(z - z.max(1, keepdims=True))
            assert np.allclose(out[:, h], e @ v[:, h // 2] / e.sum(1, keepdims=True), atol=1e-13)
            assert np.allclose(lse[:, h], np.log(np.exp(z).sum(1)), atol=1e-13)
    # window 1, one sink: the last row sees tokens 0 and 10
    out, *_ = op.attention(q[4:], k, v, 0.5, window=1, sinks=1)
    w = np.exp(0.5 * q[4, 0] @ k[[0, 10], 0].T)
    assert np.allclose(out[0, 0], w @ v[[0, 10], 0] / w.sum(), atol=1e-14)


def test_release_by_hand():
    # pages of 4: request 0 holds 10 tokens (pages 7, 3, 9), 1 holds 8 (7, 5), 2 holds 5 (1, 2)
    table = [[7, 3, 9], [7, 5, -1], [1, 2, -1]]
    shared = [0] * 10
    shared[7] = 1
    ring = [0, 4, 6, 8, -9, -9, -9, -9]
    t, g, c, s, cut = op.release([10, 8, 5], [5, 0, 5], table, ring, (8, 12), shared, 4)
    # 0 keeps 5: its third page; 1 all: page 7 is still held by 0, 5 is free
    assert t.tolist() == [[7, 3, -1], [-1, -1, -1], [1, 2, -1]]
    assert g.tolist() == [0, 4, 6, 8, 5, 9, -9, -9] and c.tolist() == [8, 14] and not s.any() and cut == []
    # both give page 7 up: free once
    t, g, c, s, cut = op.release([10, 8, 5], [0, 0, 5], table, ring, (8, 12), shared, 4)
    assert g.tolist() == [0, 4, 6, 8, 3, 5, 7, 9] and c.tolist() == [8, 16] and not s.any()
    # cut inside page 7, which request 1 holds too
    t, g, c, s, cut = op.release([10, 8, 5], [3, 8, 5], table, ring, (8, 12), shared, 4)
    assert cut == [0] and t[0].tolist() == [7, -1, -1] and s[7] == 1


def test_release_behind_a_window_by_hand():
    # 23 tokens in pages of 4, a window of 6 and 5 sinks: the next token, 23,
    # sees 18 .. 22 and 0 .. 4; tokens 5 .. 17 are passed, pages 2 and 3 wholly
    table, ring = [[0, 1, 2, 3, 4, 5]], [-9] * 6
    t, g, c, s, _ = op.release([23], [23], table, ring, (0, 0), [0] * 6, 4, 6, 5)
    assert t.tolist() == [[0, 1, -1, -1, 4, 5]] and g.tolist()[:2] == [2, 3] and c.tolist() == [0, 2]
    # again: nothing more
    t, g, c, s, _ = op.release([23], [23], t, g, c, s, 4, 6, 5)
    assert t.tolist() == [[0, 1, -1, -1, 4, 5]] and c.tolist() == [0, 2]


def test_fork_by_hand():
    table = [[3, 5, 6], [-1, -1, -1], [8, -1, -1], [-1, -1, -1]]
    c, t, s, cur, src, dst = op.fork([10, 0, 4, 0], [-1, 0, -1, 2], table, [1, 2, 4], (5, 8), [0] * 9, 4)
    assert t.tolist() == [[3, 5, 6], [3, 5, 4], [8, -1, -1], [8, -1, -1]]
    assert c.tolist() == [10, 10, 4, 4] and cur.tolist() == [6, 8]
    assert src.tolist() == [-1, 6, -1, -1] and dst.tolist() == [-1, 4, -1, -1]
    assert s.tolist() == [0, 0, 0, 1, 0, 1, 0, 0, 1]
    c, t, s, cur, src, dst = op.fork([10, 0, 4, 0], [-1, 0, -1, -1], table, [1, 2, 4], (5, 8), [0] * 9, 4, [0, 5, 0, 0])
    assert t[1].tolist() == [3, 4, -1] and c[1] == 5 and src[1] == 5 and s[5] == 0


def test_compact_by_hand():
    # held 9, 2, 7 (shared), 4; free 1, 5, 8; 0, 3 and 6 are neither
    table = [[9, 2], [7, -5], [7, 4]]
    shared = [0] * 10
    shared[7] = 1
    ring = [8, 1, 5, -3]
    t, g, s, src, dst = op.compact([8, 4, 7], table, ring, (4, 7), shared, 4)
    # in order: 1 2 4 5 | 7 8 9, so 7 and 9 move to 1 and 5
    assert src.tolist() == [7, 9, -1, -1, -1] and dst.tolist() == [1, 5, -1, -1, -1]
    assert t.tolist() == [[5, 2], [1, -5], [1, 4]]
    assert g.tolist() == [7, 8, 9, -3] and s[1] == 1 and s[7] == 0


def test_softmax_and_pick():
    assert np.allclose(ov.softmax([0.0, math.log(3.0)], 1.0), [0.25, 0.75])
    assert np.allclose(ov.softmax([0.0, math.log(3.0)], 0.5), [0.1, 0.9])
    assert ov.softmax([1.0, 2.0, 2.0], 0.0).tolist() == [0, 1, 0]
    assert ov.softmax([-math.inf, 0.0], 1.0).tolist() == [0, 1]
    for bad in ([-math.inf] * 2, [0.0, math.nan], [0.0, math.inf]):
        assert ov.softmax(bad, 1.0) is None
    assert ov.softmax([0.0], -1.0) is None and ov.softmax([0.0], math.nan) is None
    w = [0.0, 2.0, 0.0, 2.0]
    assert [ov.pick(w, u)[0] for u in (0.0, 0.49, 0.5, 0.99, 1.0, 2.0, -1.0, math.nan)] == [1, 1, 3, 3, 3, 3, 1, 1]


@pytest.mark.parametrize("certain", [False, True])
def test_answers_are_distributed_as_the_model(certain):
    # one draft of three tokens: over an even grid of its random number and the
    # other's, with the draft drawn from q, the first token follows p
    z, d = np.array([[0.3, -1.0, 1.1], [0.0, 2.0, 1.0]]), np.array([[1.0, 0.2, -0.4], [0.0, 0.0, 0.0]])
    p, q = ov.softmax(z[0], 0.7), ov.softmax(d[0], 0.7)
    n = 40
    grid = (np.arange(n) + 0.5) / n
    mass = np.zeros(3)
    for x in range(3):
        share = (1.0 / 3 if certain else q[x]) / n ** 2  # a certain drafter names each in turn
        for u in grid:
            for w in grid:
                a, token, _ = ov.request(z, [x, 0], [u, w], None if certain else d, 0.7)
                mass[x if a else token] += share
    # each of the two grids is off by 1 / 2n at most at a border, three borders
    assert np.abs(mass - p).max() <= 3 / n


def test_greedy_requests():
    z = np.array([[0.0, 5.0, 5.0], [1.0, 0.0, 0.5], [0.0, 0.0, 9.0]])
    assert ov.request(z, [1, 0, 0], [0.9, 0.9, 0.5], None, 0.0)[:2] == (2, 2)
    assert ov.request(z, [2, 0, 0], [0.0, 0.0, 0.5], None, 0.0)[:2] == (0, 1)
    assert ov.request(z, [1, 2, 0], [0.0, 0.0, 0.5], z, 0.0)[:2] == (1, 0)


def test_refused_certain_drafts_are_not_drawn_again():
    z = np.log(np.array([[0.5, 0.25, 0.25], [1.0, 1e-9, 1e-9]]))
    assert ov.request(z, [0, 0], [0.6, 0.0])[:2] == (0, 1)
    assert ov.request(z, [0, 0], [0.6, 0.5])[:2] == (0, 2)
    assert ov.request(z, [0, 0], [0.4, 0.5])[:2] == (1, 0)
    assert ov.request(z, [7, 0], [0.0, 0.6])[:2] == (0, 1)     # outside the vocabulary
    assert ov.request(np.full((1, 3), np.nan), [0], [0.5])[:2] == (0, -1)
