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
