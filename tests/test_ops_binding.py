"""What the binding of the balance loss, the matrix-vector products and the paged cache passes to the C entry points,
shown on host tensors with the launches replaced by a record of their arguments."""

import pytest
import torch

import mixed_precision_moe_amd as mx
from mixed_precision_moe_amd import ops

saved = torch.autograd.graph.saved_tensors_hooks


@pytest.fixture
def calls(monkeypatch):
    """The calls that would be launched, as (entry point, arguments); host tensors pass for GPU tensors."""
    made = []
    monkeypatch.setattr(ops, "_gpu_of", lambda name, *tensors: 0)
    monkeypatch.setattr(ops, "_call", lambda index, fn, *args: made.append((fn, args)))
    return made


def balance(T=8, E=4, pad=12, mask=False):
    logits = torch.zeros(T, E + pad)[:, :E].requires_grad_()
    ids = torch.zeros(T, 2, dtype=torch.int32)
    return logits, mx.balance_loss(logits, ids, torch.ones(T, dtype=torch.bool) if mask else None)[0]


def test_backward_of_saved_strided_logits(calls):
    logits, loss = balance()
    torch.autograd.grad(loss, logits)
    fn, args = calls[-1]
    assert fn == "moe_balance_backward" and args[:4] == (logits.data_ptr(), 8, 4, 16)


def test_backward_takes_the_rows_that_saved_tensor_hooks_return(calls):
    """Hooks may return a copy with another stride than the tensor that was saved (save_on_cpu does)."""
    given = []

    def unpack(t):
        given.append(t.contiguous())
        return given[-1]

    with saved(lambda t: t, unpack):
        logits, loss = balance()
    torch.autograd.grad(loss, logits)
    copy = next(t for t in given if t.shape == (8, 4))
    assert calls[-1][1][:4] == (copy.data_ptr(), 8, 4, 4)


@pytest.mark.parametrize("change", [
    lambda t: t.t().contiguous().t() if t.dtype == torch.float32 and t.dim() == 2 else t,  # columns apart
    lambda t: t[:1].expand(8, 4) if t.dim() == 2 else t,                                   # rows on each other
    lambda t: t.half() if t.dtype == torch.float32 else t,
    lambda t: t[:7] if t.dim() == 2 else t,
    lambda t: t[:5] if t.dtype == torch.bool else t,
    lambda t: t.repeat_interleave(2)[::2] if t.dtype == torch.bool else t])
def test_backward_refuses_other_tensors_than_were_saved(calls, change):
    with saved(lambda t: t, change):
        logits, loss = balance(mask=True)
    calls.clear()
    with pytest.raises((ValueError, RuntimeError)):
        torch.autograd.grad(loss, logits)
    assert not calls


@pytest.mark.parametrize("T,E", [(8, 4), (5000, 96), (3000, 1024)])
def test_only_the_rows_the_mask_and_d_live_until_the_backward_pass(calls, T, E):
    kept = []

    def pack(t):
        kept.append(t)
        return t

    with saved(pack, lambda t: t):
        _, loss = balance(T, E, mask=True)
    kept += [t for t in vars(loss.grad_fn).values() if torch.is_tensor(t)]
    assert {t.untyped_storage().nbytes() for t in kept} <= {4 * T * (E + 12), T, 4 * E}


def cache(v_dim=32):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    store = [u8(4, 8, 2, 32), u8(4, 8, 2, 2), u8(4, 8, 2, 16), u8(4, 8, 2, 1)]
    return mx.PagedCache(4, 8, 2, 64, v_dim, mx.FMT_MXFP4, storage=store if v_dim else store[:2] + [None, None])


def write_and_read(c, calls):
    """The cache's four addresses as the write and the read got them."""
    k, v = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 32, dtype=torch.bfloat16)
    v = v if c.v_q is not None else None
    table, cu = torch.zeros(1, 1, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32)
    c.write(k, v, table, cu)
    c.read(table, cu, k_out=k, v_out=v)
    (fw, w), (fr, r) = calls[-2:]
    assert (fw, fr) == ("mxfp4_cache_write", "mxfp4_cache_read") and w[0]._obj.num_pages == r[0]._obj.num_pages == 4
    assert w[-4:] == r[1:5]
    return w[-4:]


@pytest.mark.parametrize("v_dim", [32, 0])
def test_the_caches_memory_and_sizes_are_not_replaced(calls, v_dim):
    c = cache(v_dim)
    names = ("k_q", "k_s", "v_q", "v_s")
    for name in names:
        with pytest.raises(AttributeError):
            setattr(c, name, torch.zeros(1, 8, 2, 32, dtype=torch.uint8))
    with pytest.raises(AttributeError):
        c.dims = None
    c.dims.num_pages = 1 << 20  # of a copy
    c.dims.page_size = 1 << 10
    assert (c.dims.num_pages, c.dims.page_size) == (4, 8)
    assert write_and_read(c, calls) == tuple(t if t is None else t.data_ptr() for t in (getattr(c, n) for n in names))


def test_the_caches_addresses_are_those_at_the_call(calls):
    """Memory that moves under its tensors: given back and taken again, as an offloaded cache's is."""
    c = cache()
    old = write_and_read(c, calls)
    c.k_q.untyped_storage().resize_(0)
    assert write_and_read(c, calls)[0] == 0
    held = torch.empty(c.k_q.numel(), dtype=torch.uint8)  # what was free is likely to be here
    c.k_q.untyped_storage().resize_(c.k_q.numel())
    c.v_s.set_(torch.ones_like(c.v_s))
    new = write_and_read(c, calls)
    assert new == tuple(t.data_ptr() for t in (c.k_q, c.k_s, c.v_q, c.v_s)) and new[0] != held.data_ptr()
    assert new[1:3] == old[1:3]


WIDE = (1 << 32) + 16  # 16 in 32 bits


@pytest.mark.parametrize("kw", [dict(heads=WIDE), dict(page_size=WIDE), dict(k_dim=WIDE * 2), dict(v_dim=WIDE * 2),
                                dict(fmt=(1 << 32) + 2), dict(page_size=1 << 31), dict(heads=-WIDE)])
def test_cache_sizes_past_32_bits_are_refused(calls, kw):
    args = dict(num_pages=1, page_size=16, heads=1, k_dim=32, v_dim=0, fmt=mx.FMT_MXFP8, device="meta")
    mx.PagedCache(**args)
    with pytest.raises((ValueError, mx.Mxfp4Error)):
        mx.PagedCache(**{**args, **kw})


def test_calls_with_sizes_past_32_bits_are_refused(calls):
    z = lambda *s, d=torch.int32: torch.empty(*s, dtype=d, device="meta")  # noqa: E731
    c = mx.PagedCache(1, 16, 1, 32, 0, mx.FMT_MXFP8, device="meta")
    rows = z(3, 1, 32, d=torch.bfloat16)
    calls.clear()
    for bad in (lambda: mx.balance_loss(z(0, WIDE, d=torch.float32), z(0, 2)),
                lambda: mx.balance_loss(z(1, 64, d=torch.float32), z(1, WIDE)),
                lambda: c.write(rows, None, z(1, WIDE), z(2)), lambda: c.read(z(WIDE, 0), z(WIDE + 1), rows=3),
                lambda: mx.fp4_expert_matvec(z(0, 32, d=torch.bfloat16), z(WIDE, 1, 16, d=torch.uint8),
                                             z(WIDE, 1, 1, d=torch.uint8), z(WIDE + 1), z(0)),
                lambda: mx.fp4_expert_matvec(z(0, 32, d=torch.bfloat16), z(2, 1, 16, d=torch.uint8),
                                             z(2, 1, 1, d=torch.uint8), z(3), z(0), top_k=WIDE)):
        with pytest.raises(ValueError):
            bad()
    assert not calls
