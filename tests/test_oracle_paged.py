"""The paged operators' oracle (oracle/paged.py) against hand-worked values
and independent formulas."""
import numpy as np
import pytest

from oracle import paged as op


def test_plan_by_hand():
    # pages of 4; request 0 holds 5 tokens on pages 9 and 8, request 1 none
    table, lens, cu, slots, pos, cursor = op.plan([5, 0], [4, 5], [[9, 8, -1], [-1, -1, -1]], [3, 4, 5, 6], (6, 9), 4,
                                                  11)
    assert table.tolist() == [[9, 8, 5], [6, 3, -1]]
    assert lens.tolist() == [9, 5] and cu.tolist() == [0, 4, 9]
    assert slots.tolist() == [33, 34, 35, 20, 24, 25, 26, 27, 12, -1, -1]
    assert pos.tolist() == [5, 6, 7, 8, 0, 1, 2, 3, 4, 0, 0] and cursor.tolist() == [9, 9]


def test_plan_out_of_pages():
    table, _, _, slots, _, cursor = op.plan([0, 0], [2, 2], [[-1], [-1]], [7], (0, 1), 2, 4)
    assert table.tolist() == [[7], [-1]] and slots.tolist() == [14, 15, -1, -1] and cursor.tolist() == [1, 1]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_angles(interleaved):
    rng = np.random.default_rng(0)
    angle = np.arange(50)[:, None] * 10000.0 ** (-np.arange(0, 8, 2) / 8)
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    q, k = rng.standard_normal((2, 1, 1, 12))
    turn = lambda x, p: op.rotate(x, [p], table, interleaved)[0, 0]  # noqa: E731
    assert np.isclose(np.linalg.norm(turn(q, 37)), np.linalg.norm(q))
    assert np.array_equal(turn(q, 37)[8:], q[0, 0, 8:])
    assert np.isclose(turn(q, 30) @ turn(k, 12), turn(q, 40) @ turn(k, 22))


def test_attention_by_the_whole_matrix():
    rng = np.random.default_rng(1)
    n, s, heads, kv, dim = 5, 9, 4, 2, 6
    q, k, v = rng.standard_normal((n, heads, dim)), rng.standard_normal((s, kv, dim)), rng.standard_normal((s, kv, dim))
    for causal in (True, False):
        for window in (0, 1, 3):
            out, lse = op.attention(q, k, v, 0.7, causal, window)[:2]
            for h in range(heads):
                z = 0.7 * q[:, h] @ k[:, h // 2].T
                i, j = np.arange(s - n, s)[:, None], np.arange(s)[None, :]
                hidden = (causal & (j > i)) | ((window > 0) & (j <= i - window))
                e = np.where(hidden, 0.0, np.exp(z))
                assert np.allclose(out[:, h], e @ v[:, h // 2] / e.sum(1, keepdims=True))
                assert np.allclose(lse[:, h], np.log(e.sum(1)))


def test_attention_rows_without_keys():
    q = np.ones((3, 1, 2))
    out, lse = op.attention(q, np.ones((1, 1, 2)), np.ones((1, 1, 2)), 1.0)[:2]
    assert np.isneginf(lse[:2]).all() and (out[:2] == 0).all() and (out[2] == 1).all()
    assert np.isneginf(op.attention(q, np.ones((0, 1, 2)), np.ones((0, 1, 2)), 1.0)[1]).all()
