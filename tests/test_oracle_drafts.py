"""Pins of the oracle's attention, page pool and rotary positions against hand values, brute force and closed forms."""

import numpy as np
import pytest

from oracle import attend as A
from oracle import pages as P
from oracle import rotary as R


def test_attention_hand_values():
    # two positions with equal scores: the mean; a third that only the second draft sees
    k, v = np.zeros((4, 1, 2)), np.arange(8.0).reshape(4, 1, 2)
    q = np.ones((2, 1, 2))
    out, weight, _ = A.attend_ref(q, k, v, [0, 2], [1], [[0, 1]], 2)
    np.testing.assert_array_equal(out[:, 0], [[1, 2], [2, 3]])
    np.testing.assert_array_equal(weight, out)
    # the mask takes the first draft from the second
    out, _, _ = A.attend_ref(q, k, v, [0, 2], [1], [[0, 1]], 2, mask=[[1, 0], [0, 1]])
    np.testing.assert_array_equal(out[1, 0], [2, 3])
    # log 3 apart: weights 3/4 and 1/4
    k[0] = np.log(3.0) / 2
    out, _, score = A.attend_ref(q[:1], k, v, [0, 1], [1], [[0, 1]], 2, scale=1.0)
    np.testing.assert_allclose(out[0, 0], [0.5, 1.5])
    assert score[0, 0] == pytest.approx(np.log(3.0))


def test_attention_by_loops():
    g = np.random.default_rng(1)
    k, v, q = g.standard_normal((12, 2, 4)), g.standard_normal((12, 2, 3)), g.standard_normal((5, 4, 4))
    table, cu, start = [[3, 0, -1], [9, 2, 1]], [1, 3, 5], [2, 4]
    mask = g.random((5, 2)) < 0.5
    out, _, _ = A.attend_ref(q, k, v, cu, start, table, 3, mask)
    assert np.isnan(out[0]).all()
    for t in range(1, 5):
        b = 0 if t < 3 else 1
        for h in range(4):
            num, den = np.zeros(3), 0.0
            for pos in range(start[b] + 2):
                page = table[b][pos // 3]
                if not 0 <= page < 4 or pos >= start[b] and not mask[t, pos - start[b]]:
                    continue
                w = np.exp(0.5 * q[t, h] @ k[page * 3 + pos % 3, h // 2])
                num, den = num + w * v[page * 3 + pos % 3, h // 2], den + w
            np.testing.assert_allclose(out[t, h], num / den if den else 0.0, atol=1e-12)


def test_accepted_and_compaction():
    assert [P.accepted_ref(p) for p in ([-1], [0, 1, 2], [2, 2, 3], [0, 5, 4], [3, -1, 4], [])] == [0, 3, 1, 2, 1, 0]
    a = np.arange(8)[:, None]
    assert P.compact_ref([a], [[1, 0]], [1], [[0, 2, 4, 6]], 4, 2) == [5]
    # positions 0.. are slots 4 5 6 7 0 1 2 3; position 2 takes 3, 3 takes 5, 4 takes 7
    assert list(a[[4, 5, 6, 7, 0, 1, 2, 3], 0]) == [4, 5, 7, 1, 3, 1, 2, 3]


def test_pool_hand_values():
    refs, table = np.zeros(6, int), np.full((3, 3), -1)
    data = np.arange(12)[:, None]
    assert P.resize_ref(refs, table, [5, 0, 2], 2) == 0
    assert table.tolist() == [[0, 1, 2], [-1, -1, -1], [3, -1, -1]] and list(refs) == [1, 1, 1, 1, 0, 0]
    assert P.fork_ref(refs, table, [0], [1], [3], 2, [data]) == 0
    assert table[1].tolist() == [0, 4, -1] and list(refs) == [2, 1, 1, 1, 1, 0] and data[8, 0] == 2 and data[9, 0] == 9
    # row 1 ends inside the shared page: it gets the last free one
    assert P.resize_ref(refs, table, [-1, 1, -1], 2, [data]) == 0
    assert table[1].tolist() == [4, -1, -1] and list(refs) == [1, 1, 1, 1, 1, 0] and data[8, 0] == 0
    assert P.resize_ref(refs, table, [-1, 6, 4], 2) == 2 and table.tolist()[1:] == [[4, 5, -1], [3, -1, -1]]
    assert P.resize_ref(refs, table, [0, 0, 0], 2) == 0 and not refs.any() and (table == -1).all()


def test_rotary_closed_forms():
    assert R.turns_ref(7, 0.25) == 0.75 and R.turns_ref(-1, 0.25) == 0.75 and R.turns_ref((1 << 31) - 1, 0.5) == 0.5
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    np.testing.assert_allclose(R.rotary_ref(x, [1], [0.25, 0.5]), [[[-3, -2, 1, -4, 9]]], atol=1e-15)
    np.testing.assert_allclose(R.rotary_ref(x, [1], [0.25, 0.5], interleaved=True), [[[-2, 1, -3, -4, 9]]], atol=1e-15)
    y = R.rotary_ref(x, [3], [0.1], offset=2, magnitude=2.0)
    np.testing.assert_allclose(R.rotary_ref(y, [3], [0.1], offset=2, magnitude=0.5, inverse=True), x, atol=1e-14)
    np.testing.assert_allclose(R.frequencies_ref(4, 100.0), [1.0, 0.1])
