"""Batches whose sequences have very different numbers of rows, so that the average that tiles are chosen by fits none of them."""

import numpy as np
import pytest
import torch

from tests.test_gpu_attend import FMTS, Setup, tree_mask

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("group,k_dim,v_dim,new", [
    (4, 64, 64, [200] + [1] * 30), (4, 128, 128, [1] * 7 + [300, 0, 2]), (1, 64, 128, [1] * 40 + [90]), (8, 192, 128, [1, 150, 1, 1]),
    (2, 256, 256, [70, 1, 0, 0, 1]), (16, 64, 64, [0, 40, 1, 1, 1, 1, 1, 1])])
@pytest.mark.parametrize("tree", [False, True])
def test_chunks_beside_single_tokens(fmt, group, k_dim, v_dim, new, tree):
    g = np.random.default_rng(len(new))
    have = [int(x) for x in g.integers(0, 400, len(new))]
    s = Setup(fmt, 32, 1, k_dim, v_dim, have, new, group)
    mask = tree_mask(s.g, new, s.rows, 0) if tree else None
    s.check(s.cache.attend(s.q, *s.args(), tree_mask=None if mask is None else torch.from_numpy(mask).cuda()), mask)


def test_a_chunk_beside_long_contexts():
    s = Setup("mxfp8", 16, 1, 64, 64, [9000, 20, 5000, 0], [1, 130, 2, 33], 4)
    s.check(s.cache.attend(s.q, *s.args()))
