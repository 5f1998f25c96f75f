"""GPU parity of compaction and page copies, byte by byte, where a workgroup takes several rounds, where many share a token's
units, and for planes whose tokens start on 1, 2, 4, 8 and 16 bytes."""

import numpy as np
import pytest

from mixed_precision_moe_amd import synth
from oracle import pages as P
from tests.test_gpu_pages import i32, make, same

pytestmark = pytest.mark.gpu


def test_compaction_in_rounds():
    """So many sequences that one workgroup has all units of a sequence, more than a round's."""
    B, W, page = 4200, 24, 16
    g = synth.rng(361)
    c, planes, g = make("mxfp8", 2 * B, page, 8, 128, 64)
    table = g.permutation(2 * B).reshape(B, 2).astype(np.int32)
    start = g.integers(0, 2 * page - W + 1, B).astype(np.int32)
    path = np.full((B, W), -1, np.int32)
    for b in range(B):
        n = (b * 7) % (W + 1)
        path[b, :n] = np.sort(g.permutation(W)[:n])
    want = P.compact_ref(planes, table, start, path, page, 2 * B)
    assert c.compact(i32(table), i32(start), i32(path)).tolist() == want
    same(c, planes)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
@pytest.mark.parametrize("heads,k_dim,v_dim", [(64, 256, 128), (1, 32, 64), (2, 32, 32), (3, 32, 96), (5, 96, 0)])
@pytest.mark.parametrize("odd", [False, True])
def test_compaction_in_stripes(fmt, heads, k_dim, v_dim, odd):
    W, page = 60, 8
    c, planes, g = make(fmt, 24, page, heads, k_dim, v_dim, seed=heads, odd=odd)
    table = g.permutation(24).reshape(2, 12).astype(np.int32)
    start = np.array([3, 21], np.int32)
    path = np.full((2, W), -1, np.int32)
    path[0, :40] = np.sort(g.permutation(W)[:40])
    path[1] = np.arange(1, W + 1)  # each where the next one goes
    want = P.compact_ref(planes, table, start, path, page, 24)
    assert c.compact(i32(table), i32(start), i32(path)).tolist() == want
    same(c, planes)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
@pytest.mark.parametrize("page,heads,k_dim,v_dim,odd", [(200, 16, 256, 128, False), (37, 3, 96, 32, True), (1, 1, 32, 0, False), (64, 8, 128, 128, False)])
def test_large_and_small_pages_copied(fmt, page, heads, k_dim, v_dim, odd):
    c, planes, g = make(fmt, 12, page, heads, k_dim, v_dim, odd=odd)
    src, dst, rows = [0, 1, 2, 3, 4], [6, 7, 8, 9, 10], [page, page - 1, 1, page // 2, -5]
    for s, d, r in zip(src, dst, rows):
        for a in planes:
            a[d * page:d * page + max(r, 0)] = a[s * page:s * page + max(r, 0)]
    c.copy_pages(i32(src), i32(dst), i32(rows))
    same(c, planes)
