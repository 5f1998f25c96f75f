"""NaN in queries and in what they see gives NaN in those rows' results, and in no others, however the context is split."""

import numpy as np
import pytest
import torch

from oracle import attend as A
from tests.gpu_common import bf16_host_f64
from tests.test_gpu_attend import FMTS, Setup, tolerance

pytestmark = pytest.mark.gpu

# few rows and many (up to 16, 32, 64, 128 and 256 rows a tile), contexts in one piece, in a few parts and in many
SIZES = [(2, 4, 64, 64, [60], [1]), (1, 2, 64, 64, [9000, 3, 2500], [2, 1, 5]), (1, 8, 128, 128, [30000], [4]), (2, 8, 64, 128, [7000, 20], [7, 3]),
         (1, 8, 192, 128, [3000, 400], [33, 9]), (1, 8, 128, 128, [700], [150]), (1, 2, 256, 256, [5000], [3]), (1, 4, 256, 224, [2000], [40])]


def clean(s, scale=None):
    with np.errstate(all="ignore"):
        out, weight, score = A.attend_ref(bf16_host_f64(s.q), *s.values(), s.cu, s.have, s.table, s.page, scale=scale)
    return out, tolerance(out, weight, score, s.q.shape[2], max(s.have) + max(s.new), 2.0 ** -8)


def agrees(got, out, tol, nan):
    got = got.double().cpu().numpy()
    assert np.isnan(got[nan]).all()
    assert np.all(np.abs(got - out)[~nan] <= tol[~nan])


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("heads,group,k_dim,v_dim,have,new", SIZES)
def test_a_query_that_is_not_a_number(fmt, heads, group, k_dim, v_dim, have, new):
    s = Setup(fmt, 32, heads, k_dim, v_dim, have, new, group)
    out, tol = clean(s)
    agrees(s.cache.attend(s.q, *s.args()), out, tol, np.zeros(out.shape, bool))
    nan = np.zeros(out.shape, bool)
    for row, head, i in ((0, 1, 0), (s.rows - 1, heads * group - 1, k_dim - 1)):
        s.q[row, head, i] = float("nan")
        nan[row, head] = True
    agrees(s.cache.attend(s.q, *s.args()), out, tol, nan)


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("heads,group,k_dim,v_dim,have,new", SIZES)
@pytest.mark.parametrize("plane", ["k", "v"])
def test_a_context_position_that_is_not_a_number(fmt, heads, group, k_dim, v_dim, have, new, plane):
    s = Setup(fmt, 32, heads, k_dim, v_dim, have, new, group)
    out, tol = clean(s)
    pos, block = have[0] // 2, 16 if fmt == "nvfp4" else 32
    page, slot = s.table[0, pos // 32], pos % 32
    nan = np.zeros(out.shape, bool)
    rows = slice(0, new[0])  # of the first sequence, and the query heads of key head 0
    if fmt == "mxfp8":
        getattr(s.cache, plane + "_q")[page, slot, 0, 1] = 0x7F
        hit = slice(1, 2)
    else:  # a scale that is no number
        getattr(s.cache, plane + "_s")[page, slot, 0, 1] = 0x7F if fmt == "nvfp4" else 0xFF
        hit = slice(block, 2 * block)
    nan[rows, :group, slice(None) if plane == "k" else hit] = True
    agrees(s.cache.attend(s.q, *s.args()), out, tol, nan)


@pytest.mark.parametrize("group", [2, 40, 200])
@pytest.mark.parametrize("pos", [5, 4500, 8990])
def test_a_value_that_is_not_a_number_under_no_weight(group, pos):
    """Scores so far apart that most positions, and most parts of the context, weigh nothing beside the best."""
    s = Setup("mxfp8", 32, 1, 64, 64, [9000], [1], group)
    out, tol = clean(s, 200.0)
    nan = np.zeros(out.shape, bool)
    nan[:, :, 7] = True
    s.cache.v_q[s.table[0, pos // 32], pos % 32, 0, 7] = 0x7F
    got = s.cache.attend(s.q, *s.args(), scale=200.0)
    if pos > 8960 and bool(torch.isnan(got).all()):
        return  # beside drafts, whose values are not looked at in part, all of the result may be NaN: at least the element is
    agrees(got, out, tol, nan)
