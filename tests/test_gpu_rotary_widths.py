"""GPU parity of the rotary positions where accesses of 16, 8, 4 and fewer bytes are taken, with and without elements beside
the turned ones, with one tensor and two, in place and not.  The tolerance is that of test_gpu_rotary.py."""

import pytest
import torch

import mixed_precision_moe_amd as mx
from tests.test_gpu_rotary import close, i32, make, spread

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,dim,rot,offset", [
    (5, 3, 128, 64, 64), (4, 7, 128, 64, 32), (6, 5, 96, 40, 8), (3, 2, 72, 24, 4), (9, 4, 68, 36, 12), (5, 300, 20, 12, 4), (3, 3, 22, 10, 2),
    (4, 2, 21, 8, 3), (513, 1, 64, 2, 6), (2, 130, 6, 6, 0)])
def test_widths(dtype, interleaved, rows, heads, dim, rot, offset):
    q, k, p = make(rows, heads, dim, dtype), make(rows, 1, dim, dtype, 1), spread(rows)
    r = mx.Rotary(rot, interleaved=interleaved, offset=offset)
    for second in (k, None):
        qo, ko = r(q, second, i32(p))
        close(qo, q, p, r)
        if second is None:
            assert ko is None
        else:
            close(ko, second, p, r)
    before = q.clone()
    out, none = r(q, None, i32(p), inplace=True)
    assert out is q and none is None
    close(q, before, p, r)
