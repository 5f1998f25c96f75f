"""What the binding of the attention over the cache, compaction, the page pool and rotary positions passes to the C entry
points, and what it refuses, shown on host tensors with the launches replaced by a record of their arguments."""

import math

import pytest
import torch

import mixed_precision_moe_amd as mx
from mixed_precision_moe_amd import ops, rotary

WIDE = (1 << 32) + 16  # 16 in 32 bits


@pytest.fixture
def calls(monkeypatch):
    """The calls that would be launched, as (entry point, arguments); host tensors pass for GPU tensors."""
    made = []
    for module in (ops, rotary):
        monkeypatch.setattr(module, "_gpu_of", lambda name, *tensors: 0)
        monkeypatch.setattr(module, "_call", lambda index, fn, *args: made.append((fn, args)))
    return made


def cache(v_dim=32, pages=4):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    store = [u8(pages, 8, 2, 32), u8(pages, 8, 2, 2), u8(pages, 8, 2, 16), u8(pages, 8, 2, 1)]
    return mx.PagedCache(pages, 8, 2, 64, v_dim, mx.FMT_MXFP4, storage=store if v_dim else store[:2] + [None, None])


def i32(*a):
    return torch.tensor(a, dtype=torch.int32)


def test_host_tensors_are_refused():
    rot = mx.Rotary(32, device="cpu")
    with pytest.raises(ValueError, match="GPU tensor"):
        rot(torch.zeros(3, 1, 32), None, i32(0, 1, 2))


def test_attention_arguments(calls):
    c = cache()
    q, table, cu = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32), i32(0, 3)
    out = c.attend(q, table, cu)
    fn, a = calls[-1]
    assert fn == "mxfp4_cache_attend" and a[1:5] == tuple(t.data_ptr() for t in (c.k_q, c.k_s, c.v_q, c.v_s))
    assert a[5:10] == (q.data_ptr(), 256, 64, 4, 3) and out.shape == (3, 4, 32) and out.dtype == torch.bfloat16
    assert a[16] is None and a[19] == 64 ** -0.5 and a[20:24] == (out.data_ptr(), 128, 32, 0)
    # a mask of no columns hides all drafts and is no absent mask
    c.attend(q, table, cu, tree_mask=torch.zeros(3, 0, dtype=torch.bool))
    assert calls[-1][1][16] and calls[-1][1][18] == 0
    mask = torch.zeros(3, 9, dtype=torch.bool)
    c.attend(q, table, cu, tree_mask=mask[:, 2:6], scale=2.0, out_dtype=torch.float32)
    assert calls[-1][1][16:20] == (mask.data_ptr() + 2, 9, 4, 2.0) and calls[-1][1][23] == 1
    # the strides of one row and of one head say nothing
    one = torch.zeros(1, 4, 64, dtype=torch.bfloat16).as_strided((1, 4, 64), (7, 64, 1))
    c.attend(one, table, i32(0, 1))
    assert calls[-1][1][6:8] == (256, 64)


def test_sizes_past_32_bits_are_refused(calls):
    z = lambda *s, d=torch.int32: torch.empty(*s, dtype=d, device="meta")  # noqa: E731
    c = mx.PagedCache(1, 16, 1, 32, 32, mx.FMT_MXFP8, device="meta")
    q = z(3, 1, 32, d=torch.bfloat16)
    pool = mx.PagePool(c)
    rot = mx.Rotary(2, device="cpu")
    calls.clear()
    for bad in (lambda: c.attend(q, z(1, WIDE), z(2)), lambda: c.attend(q, z(1, 1), z(2), tree_mask=z(3, WIDE, d=torch.bool)),
                lambda: c.attend(z(0, WIDE, 32, d=torch.bfloat16), z(1, 1), z(2)),
                lambda: c.compact(z(WIDE, 0), z(WIDE), z(WIDE, 0)), lambda: c.compact(z(1, 1), z(1), z(1, WIDE)),
                lambda: c.copy_pages(z(WIDE), z(WIDE)), lambda: pool.resize(z(WIDE, 1), z(WIDE)), lambda: pool.resize(z(1, WIDE), z(1)),
                lambda: pool.fork(z(1, 1), z(WIDE), z(WIDE), z(WIDE)), lambda: pool.resize(z(1 << 16, 1 << 15), z(1 << 16)),
                lambda: rot(z(0, WIDE, 2, d=torch.float32), None, z(0)), lambda: rot(z(0, 1, WIDE, d=torch.float32), None, z(0)),
                lambda: rot(z(0, 1, 2, d=torch.float32), z(0, WIDE, 2, d=torch.float32), z(0))):
        with pytest.raises(ValueError):
            bad()
    assert not calls


def test_a_pool_copies_in_all_its_caches(calls):
    a, b = cache(), cache(0)
    pool = mx.PagePool(a, b, refs=torch.zeros(4, dtype=torch.int32))
    table = torch.full((3, 5), -1, dtype=torch.int32)
    missing = pool.resize(table, i32(9, 0, 3))
    (f0, r), (f1, x), (f2, y) = calls
    assert (f0, f1, f2) == ("mxfp4_pool_resize", "mxfp4_cache_copy_pages", "mxfp4_cache_copy_pages")
    assert r[:2] == (4, 8) and r[2] == pool.refs.data_ptr() and r[3:7] == (table.data_ptr(), 5, 3, 5)
    copies = r[8]
    assert r[9] == missing.data_ptr() and missing.shape == () and copies == r[10] + r[11]
    assert x[1:5] == y[1:5] == (copies, copies + 12, copies + 24, 3)
    assert x[5] == a.k_q.data_ptr() and y[5] == b.k_q.data_ptr() and y[7] is None
    with pytest.raises(AttributeError):
        pool.refs = torch.zeros(1 << 20, dtype=torch.int32)
    with pytest.raises(AttributeError):
        pool.caches = ()
    with pytest.raises(ValueError, match="same number of pages"):
        mx.PagePool(a, cache(pages=5))


def test_rotary_arguments_and_gradients(calls):
    rot = mx.Rotary(32, offset=16, interleaved=True, device="cpu", scaling=dict(kind="ramp", factor=16.0, length=8192))
    packed = torch.zeros(3, 8, 64)
    q, k = packed[:, :4].detach().requires_grad_(), packed[:, 4:6].detach().requires_grad_()
    qo, ko = rot(q, k, i32(0, 1, 2))
    fn, a = calls[-1]
    assert fn == "mxfp4_rotary" and a[2:10] == (3, 64, 32, 16, 1, 1.0 + 0.1 * math.log(16.0), 0, 1)
    assert a[10:14] == (q.data_ptr(), 512, 64, 4) and a[15:17] == (256, 64) and a[17:21] == (k.data_ptr(), 512, 64, 2)
    torch.autograd.grad((qo, ko), (q, k), (torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)))
    assert calls[-1][1][8] == 1 and calls[-1][1][13] == 4 and calls[-1][1][20] == 2
    qo, ko = rot(q, k, i32(0, 1, 2))
    torch.autograd.grad(ko.sum(), k)  # an expanded gradient of the keys alone
    a = calls[-1][1]
    assert a[8] == 1 and a[13] == 2 and a[17] is None
    # saved positions that changed since
    p = i32(0, 1, 2)
    qo, _ = rot(q, None, p)
    p.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(qo.sum(), q)


def test_frequencies():
    f, m = mx.rotary_frequencies(64)
    assert f.dtype == torch.float64 and m == 1.0 and f[0] == 1.0
    assert float(f[16]) == pytest.approx(0.01, rel=1e-14)
    assert torch.equal(mx.rotary_frequencies(64, scaling=dict(kind="linear", factor=4.0))[0], f / 4)
    g, _ = mx.rotary_frequencies(64, scaling=dict(kind="base", factor=8.0))
    assert float(g[0]) == 1.0 and float(g[31]) == pytest.approx(float(f[31]) / 8, rel=1e-12)
    # 64 pairs, base 10000, 8192 positions: pair i turns 8192 / (2 pi) 10000^(-i / 64) times: 32 times at i = 25.8, once at 49.8
    g, m = mx.rotary_frequencies(128, scaling=dict(kind="ramp", factor=16.0, length=8192))
    f = mx.rotary_frequencies(128)[0]
    assert m == pytest.approx(1.2772588722239782) and torch.equal(g[:26], f[:26])
    assert torch.allclose(g[50:], f[50:] / 16, rtol=1e-15) and bool((g[26:50] <= f[26:50]).all())
    x = 13 / 25  # the ramp runs from 25 to 50
    assert float(g[38]) == pytest.approx(float(f[38]) * (1 - x + x / 16), rel=1e-13)
    g, m = mx.rotary_frequencies(128, scaling=dict(kind="bands", factor=8.0, length=8192))
    turns = 8192 * f / (2 * math.pi)
    assert m == 1.0 and torch.equal(g[turns >= 4], f[turns >= 4])
    assert torch.allclose(g[turns <= 1], f[turns <= 1] / 8, rtol=1e-14)
    for bad in (dict(dim=7), dict(dim=0), dict(dim=8, base=0.0), dict(dim=8, scaling=dict(kind="other")),
                dict(dim=8, scaling=dict(kind="linear", factor=0.0)), dict(dim=8, scaling=dict(kind="linear", factor=2.0, length=5)),
                dict(dim=2, scaling=dict(kind="base", factor=2.0)),
                dict(dim=8, scaling=dict(kind="bands", factor=2.0, length=10, low=4.0, high=4.0))):
        with pytest.raises(ValueError):
            mx.rotary_frequencies(**bad)
    for bad in (dict(dim=2050), dict(dim=8, offset=-1), dict(dim=8, freqs=[1.0]), dict(dim=8, magnitude=float("inf")),
                dict(dim=8, freqs=[1.0] * 4, scaling=dict(kind="linear", factor=2.0))):
        with pytest.raises(ValueError):
            mx.Rotary(device="cpu", **bad)
