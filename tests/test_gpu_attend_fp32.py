"""Results in fp32 of the attention over the paged cache, to what binary32 sums leave of them.

Tolerance, per element: a weight is two bf16 terms, the second off by 2^-8 of at most 2^-8 of it: 2^-16 of the weight in the
sum of values and in the sum of weights; the exponents' errors as for bf16 results (products, scaling, maximum, exponential,
in both sums); sums over twice as many terms, 2^-23 of the magnitudes each; a few roundings of the result (the reciprocal, its
product, the global scale)."""

import numpy as np
import pytest
import torch

from oracle import attend as A
from tests.gpu_common import bf16_host_f64
from tests.test_gpu_attend import FMTS, Setup, tree_mask

pytestmark = pytest.mark.gpu


def check(s, mask=None, scale=None):
    m = None if mask is None else torch.from_numpy(mask).cuda()
    got = s.cache.attend(s.q, *s.args(), tree_mask=m, scale=scale, out_dtype=torch.float32)
    with np.errstate(all="ignore"):
        out, weight, score = A.attend_ref(bf16_host_f64(s.q), *s.values(), s.cu, s.have, s.table, s.page, mask, scale)
    dim, seen = s.q.shape[2], max(s.have) + max(s.new)
    exponent = (score * (1.5 * dim + 4) * 2.0 ** -24 + 2.0 ** -22)[..., None]
    tol = (weight + np.abs(out)) * (2.0 ** -16 * (1 + 2.0 ** -7) + exponent) + weight * 2 * seen * 2.0 ** -23 + np.abs(out) * 2.0 ** -22 + 1e-30
    off = np.abs(got.double().cpu().numpy() - out)
    assert np.all(off <= tol), float(np.max(off / tol))
    # and the bf16 results are those of the other kernels
    b = s.cache.attend(s.q, *s.args(), tree_mask=m, scale=scale)
    assert bool(((b.float() - got).abs() <= torch.from_numpy(weight).cuda() * 2.0 ** -7 + got.abs() * 2.0 ** -7 + 1e-30).all())


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("page,heads,group,k_dim,v_dim,have,new", [
    (16, 2, 4, 64, 64, [77], [1]), (32, 4, 2, 64, 64, [300, 5], [1, 3]), (24, 1, 16, 128, 128, [31, 0, 200], [1, 1, 1]),
    (64, 3, 5, 96, 160, [63, 64, 129], [4, 2, 5]), (32, 2, 8, 192, 128, [300, 5], [3, 4]), (7, 5, 2, 256, 224, [130, 0, 1], [3, 20, 0]),
    (128, 1, 1, 256, 256, [500], [20]), (16, 2, 4, 128, 128, [40, 9], [12, 10]), (32, 1, 8, 64, 64, [200], [12]),
    (32, 1, 8, 192, 128, [300, 70], [9, 7]), (64, 1, 4, 256, 256, [100], [20]), (16, 1, 8, 128, 128, [256], [150]),
    (16, 1, 8, 64, 64, [100], [130]), (16, 1, 8, 192, 128, [100], [129])])
def test_rows_up_to_their_own_position(fmt, page, heads, group, k_dim, v_dim, have, new):
    check(Setup(fmt, page, heads, k_dim, v_dim, have, new, group))


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("new,group", [([5, 2, 9], 1), ([33, 0, 12], 3), ([40, 3], 8)])
def test_trees_and_scales(fmt, new, group):
    s = Setup(fmt, 24, 2, 128, 64, [100, 40, 0][:len(new)], new, group)
    check(s, tree_mask(s.g, new, s.rows, 0), -0.5)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_parts_that_are_joined(fmt):
    check(Setup(fmt, 64, 1, 64, 64, [2000, 3], [2, 1], 2))


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("page,heads,group,k_dim,v_dim,have,new", [
    (16, 2, 4, 64, 64, [77], [1]), (32, 4, 2, 64, 64, [300, 5], [1, 3]), (64, 3, 5, 96, 160, [63, 64, 129], [1, 2, 3]),
    (32, 2, 8, 192, 128, [300, 5], [1, 2]), (64, 1, 1, 256, 256, [500], [16])])
def test_few_rows_in_bf16_lose_no_more_than_their_rounding(fmt, page, heads, group, k_dim, v_dim, have, new):
    """Up to 16 rows a key head: the bf16 result is the fp32 one, rounded once."""
    s = Setup(fmt, page, heads, k_dim, v_dim, have, new, group)
    check(s)
    fine = s.cache.attend(s.q, *s.args(), out_dtype=torch.float32)
    assert torch.equal(s.cache.attend(s.q, *s.args()), fine.bfloat16())
