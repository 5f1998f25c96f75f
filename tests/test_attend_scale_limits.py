"""Which scales the attention over the cache takes, asked of its entry point without rows: no launch."""

import ctypes

import pytest

from mixed_precision_moe_amd import _lib, ops

BIG = 3.4028234663852886e38


@pytest.mark.parametrize("fmt,gs,scale,taken", [
    (ops.FMT_MXFP8, 1.0, 0.69 * BIG, True), (ops.FMT_MXFP8, 1.0, 0.7 * BIG, False), (ops.FMT_MXFP8, 1.0, -0.7 * BIG, False),
    (ops.FMT_MXFP4, 1e-38, 10.0, True), (ops.FMT_NVFP4, 1e-38, 1.0, True), (ops.FMT_NVFP4, 1e-38, -10.0, False),
    (ops.FMT_NVFP4, 1e38, BIG / 2, True), (ops.FMT_MXFP8, 1.0, float("nan"), False), (ops.FMT_MXFP8, 1.0, float("-inf"), False),
    (ops.FMT_NVFP4, 2.0 ** 127, 2.0 ** -149, True), (ops.FMT_MXFP8, 1.0, 0.0, True)])
def test_scales(fmt, gs, scale, taken):
    dims = ops.CacheDims(fmt, 1, 32, 32, 4, 0, gs, 1.0)
    status = _lib.lib().mxfp4_cache_attend(ctypes.byref(dims), *[None] * 5, 32, 32, 1, 0, None, None, None, 1, 1, 1, None, 0, 0, scale, None,
                                           32, 32, 0, None, 0, None)
    assert (status == 0) is taken
