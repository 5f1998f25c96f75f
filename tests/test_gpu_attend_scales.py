"""Scales of the scores near the ends of binary32: far below the smallest normal number, by themselves or through a large
global scale of the keys, and too large to be multiplied with."""

import numpy as np
import pytest
import torch

import mixed_precision_moe_amd as mx
from tests import test_gpu_attend as T
from tests.gpu_common import bf16_dev, bf16_host_f64
from mixed_precision_moe_amd import synth

pytestmark = pytest.mark.gpu


def times(q, power):
    return bf16_dev(synth.to_bf16_bits(bf16_host_f64(q) * 2.0 ** power))


@pytest.mark.parametrize("new,group", [([3], 2), ([20], 4)])
@pytest.mark.parametrize("power,scale", [(120, 2.0 ** -130), (120, 2.0 ** -135), (100, -2.0 ** -126), (0, 2.0 ** -149)])
def test_small_scales(new, group, power, scale):
    s = T.Setup("mxfp8", 16, 2, 64, 64, [2], new, group)
    s.q = times(s.q, power)
    s.check(s.cache.attend(s.q, *s.args(), scale=scale, out_dtype=torch.float32), scale=scale, half_step=2.0 ** -24)


@pytest.mark.parametrize("new,group", [([3], 2), ([20], 4)])
@pytest.mark.parametrize("scale", [None, 2.0 ** -6, 2.0 ** -10])
def test_large_global_scales(monkeypatch, new, group, scale):
    s = T.Setup("nvfp4", 16, 2, 64, 64, [2], new, group)
    c = s.cache
    gs = 2.0 ** 126, 77.5
    s.cache = mx.PagedCache(c.dims.num_pages, 16, 2, 64, 64, mx.FMT_NVFP4, *gs, storage=(c.k_q, c.k_s, c.v_q, c.v_s))
    monkeypatch.setitem(T.GS, "nvfp4", gs)
    s.q = times(s.q, 112)
    s.check(s.cache.attend(s.q, *s.args(), scale=scale, out_dtype=torch.float32), scale=scale, half_step=2.0 ** -24)


def test_scales_too_large_to_multiply_with():
    big = float(np.finfo(np.float32).max)
    q, t, cu = torch.zeros(1, 1, 32, dtype=torch.bfloat16, device="cuda"), T.i32([[0]]), T.i32([0, 1])
    c = mx.PagedCache(1, 4, 1, 32, 32, mx.FMT_MXFP8)
    for scale in (big, -big, 0.7 * big):
        with pytest.raises(mx.Mxfp4Error):
            c.attend(q, t, cu, scale=scale)
    assert not c.attend(q, t, cu, scale=0.69 * big).any()  # of log2 e times it there is a number
    small = mx.PagedCache(1, 4, 1, 32, 32, mx.FMT_NVFP4, 1e-38, 1.0)
    assert not small.attend(q, t, cu, scale=1.0).any()
    with pytest.raises(mx.Mxfp4Error):
        small.attend(q, t, cu, scale=10.0)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("have,new,group", [([9000, 40], [1, 2], 4), ([9000], [8], 3), ([3000], [60], 4)])
def test_values_up_to_the_bound(fmt, have, new, group):
    s = T.Setup(fmt, 32, 1, 64, 64, have, new, group)
    s.cache.v_s.copy_((s.cache.v_s.int() + 84).clamp(max=254))
    held = torch.from_numpy(s.values()[1][np.concatenate([32 * row[row >= 0] for row in s.table])])
    assert 2.0 ** 84 < float(held.abs().max()) < 2.0 ** 88
    got = s.cache.attend(s.q, *s.args(), out_dtype=torch.float32)
    assert bool(torch.isfinite(got).all())
    s.check(got, half_step=2.0 ** -24)
