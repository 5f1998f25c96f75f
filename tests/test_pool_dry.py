"""A page pool that runs dry where rows end inside pages they share: no row is left on a page that another one reads."""

import numpy as np
import pytest
import torch

from oracle import pages as P
from tests.test_gpu_pages import Pool, i32


def test_oracle_hand_values():
    # three rows hold page 1; two of them end inside it, no page is free: both let go, the third keeps it
    refs, table = np.array([3, 3]), np.array([[0, 1], [0, 1], [0, 1]])
    assert P.resize_ref(refs, table, [3, 3, -1], 2) == 2
    assert table.tolist() == [[0, -1], [0, -1], [0, 1]] and list(refs) == [3, 1]
    # all of its rows end inside it: the last one has it for itself
    refs, table = np.array([3, 3]), np.array([[0, 1], [0, 1], [0, 1]])
    assert P.resize_ref(refs, table, [3, 3, 3], 2) == 2
    assert table.tolist() == [[0, -1], [0, -1], [0, 1]] and list(refs) == [3, 1]
    # one page is free: the first row gets it, the second is alone on its own
    refs, table, data = np.array([2, 2, 0]), np.array([[0, 1], [0, 1]]), np.arange(6)[:, None]
    assert P.resize_ref(refs, table, [3, 3], 2, [data]) == 0
    assert table.tolist() == [[0, 2], [0, 1]] and list(refs) == [2, 1, 1] and data[4, 0] == 2


@pytest.mark.gpu
def test_a_row_that_got_no_copy_writes_nowhere():
    p = Pool(3, 4, 2, 3)
    p.resize([10, 0])
    p.fork([0], [1], [8])  # two whole pages, no page is left
    assert p.resize([-1, 6]) == 1
    assert p.table.tolist() == [[0, 1, 2], [0, -1, -1]] and list(p.refs) == [2, 1, 1]
    c = p.caches[0]
    x = torch.randn(2, 2, 32, device="cuda").bfloat16(), torch.randn(2, 2, 64, device="cuda").bfloat16()
    c.write(*x, p.dev[1:].contiguous(), i32([0, 2]), i32([6]))  # the row's next two tokens
    p.check(torch.tensor(0), 0)  # every byte as it was
    assert p.resize([0, 6]) == 0  # room again
    assert p.table.tolist() == [[-1, -1, -1], [0, 1, -1]]


@pytest.mark.gpu
@pytest.mark.parametrize("free", [0, 1, 2, 3])
def test_the_last_row_of_a_page_keeps_it(free):
    p = Pool(2 + free, 4, 4, 2)
    p.resize([8, 0, 0, 0])
    p.fork([0, 0, 0], [1, 2, 3], [8, 8, 8])
    assert p.resize([7, 5, 6, 7]) == 3 - free
    kept = [r for r in range(4) if p.table[r, 1] == 1]
    assert kept == ([3] if free <= 3 else []) and p.refs[1] == 1 and p.refs[0] == 4
    assert len({int(e) for e in p.table[:, 1] if e >= 0}) == free + 1


@pytest.mark.gpu
@pytest.mark.parametrize("rows,families,spare", [(1500, 200, 30), (40, 9, 0), (3000, 700, 100)])
def test_many_rows_share_few_pages(rows, families, spare):
    """Rows in families that share whole pages; members end inside them, with fewer free pages than members."""
    g = np.random.default_rng(rows)
    for alone in (0.0, 0.1, 0.5):  # rows that are left alone
        first = np.zeros(rows, int)
        first[:families] = g.integers(1, 11, families)
        pages = int((-(-first // 2)).sum()) + spare
        p = Pool(pages, 2, rows, 5)
        assert p.resize(first) == 0
        src = g.integers(0, families, rows - families)
        p.fork(src, np.arange(families, rows), [int(first[s]) // 2 * 2 for s in src])
        want = np.array([max(0, int(first[r if r < families else src[r - families]]) // 2 * 2 - g.integers(0, 2)) for r in range(rows)])
        missing = p.resize(np.where(g.random(rows) < alone, -1, want))
        assert missing > 0
        np.testing.assert_array_equal(np.bincount(p.table[p.table >= 0], minlength=pages), p.refs)
        p.resize(np.zeros(rows, int))
        assert not p.refs.any()
