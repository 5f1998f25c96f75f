"""What the binding of rotary positions and of the attention over the cache tells autograd, shown on host tensors with the
launches replaced by a record of their arguments."""

import pytest
import torch

import mixed_precision_moe_amd as mx
from tests.test_drafts_binding import cache, calls, i32  # noqa: F401  (a fixture)


def saved(x):
    """A result whose backward pass needs x as it is now."""
    w = torch.ones_like(x, requires_grad=True)
    return (w * x).sum()


@pytest.mark.parametrize("which", ["q", "k"])
def test_turning_in_place_is_seen_by_autograd(calls, which):  # noqa: F811
    rot, p = mx.Rotary(32, device="cpu"), i32(0, 1, 2)
    q, k = torch.zeros(3, 2, 32), torch.zeros(3, 1, 32)
    loss = saved(q if which == "q" else k)
    rot(q, k, p)  # out of place: nothing changes
    assert q._version == 0 and k._version == 0
    rot(q.detach(), k.detach(), p, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    loss = saved(q)
    with torch.no_grad():
        rot(q, None, p, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        x = torch.zeros(3, 2, 32)
        rot(x, None, p, inplace=True)


def test_given_results_are_seen_by_autograd(calls):  # noqa: F811
    c = cache()
    table, cu = torch.zeros(1, 2, dtype=torch.int32), i32(0, 3)
    bf16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    out, k, v = bf16(3, 4, 32), bf16(3, 2, 64), bf16(3, 2, 32)
    calls_of = (lambda: c.attend(bf16(3, 4, 64), table, cu, out=out), lambda: c.read(table, cu, k_out=k, v_out=v),
                lambda: c.read(table, cu, k_out=k, v_out=v))
    for call, t in zip(calls_of, (out, k, v)):
        loss = saved(t)
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    y = bf16(4, 16)
    loss = saved(y)
    mx.fp4_expert_matvec(bf16(4, 32), torch.zeros(1, 16, 16, dtype=torch.uint8), torch.zeros(1, 16, 1, dtype=torch.uint8), i32(0, 4),
                         i32(0, 1, 2, 3), y=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("which", ["q", "k", "both"])
@pytest.mark.parametrize("how", ["plain", "inplace", "requires_grad"])
def test_tangents_of_forward_mode_are_refused(calls, which, how):  # noqa: F811
    import torch.autograd.forward_ad as fw
    rot, p = mx.Rotary(32, device="cpu"), i32(0, 1, 2)
    q, k = torch.zeros(3, 2, 32), torch.zeros(3, 1, 32)
    with fw.dual_level():
        if which != "k":
            q = fw.make_dual(q, torch.ones_like(q))
        if which != "q":
            k = fw.make_dual(k, torch.ones_like(k))
        if how == "requires_grad":
            q.requires_grad_()
        with pytest.raises(ValueError, match="forward-mode"):
            rot(q, k, p, inplace=how == "inplace")
        rot(torch.zeros(3, 2, 32), torch.zeros(3, 1, 32), p)  # nothing to lose
    assert len(calls) == 1


def test_tangents_of_the_attention_and_of_a_backward_pass_are_refused(calls):  # noqa: F811
    import torch.autograd.forward_ad as fw
    c = cache()
    q, table, cu = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32), i32(0, 3)
    with fw.dual_level(), torch.no_grad():
        for out in (None, torch.zeros(3, 4, 32, dtype=torch.bfloat16)):
            with pytest.raises(ValueError, match="forward-mode"):
                c.attend(fw.make_dual(q, torch.ones_like(q)), table, cu, out=out)
    assert not calls
    c.attend(q, table, cu)
    rot, x = mx.Rotary(32, device="cpu"), torch.zeros(3, 2, 32, requires_grad=True)
    y, _ = rot(x, None, i32(0, 1, 2))
    with fw.dual_level():
        with pytest.raises(ValueError, match="forward-mode"):
            torch.autograd.grad(y, x, fw.make_dual(torch.ones_like(y), torch.ones_like(y)))


def test_function_transforms_are_not_passed_by(calls):  # noqa: F811
    """torch.func's wrapped tensors have no memory of their own: every transform ends in an error, none in a lost derivative."""
    rot, p = mx.Rotary(32, device="cpu"), i32(0, 1, 2)
    x = torch.zeros(3, 2, 32)
    for transform in (lambda f: torch.func.jvp(f, (x,), (x,)), lambda f: torch.func.grad(lambda y: f(y).sum())(x),
                      lambda f: torch.func.vmap(f)(x[None])):
        with pytest.raises((ValueError, RuntimeError)):
            transform(lambda y: rot(y, None, p)[0])


def test_only_what_asks_for_a_gradient_gets_one(calls):  # noqa: F811
    rot, p = mx.Rotary(32, device="cpu"), i32(0, 1, 2)
    q, k = torch.zeros(3, 2, 32, requires_grad=True), torch.zeros(3, 1, 32)
    for a, b in ((q, k), (k, q)):
        calls.clear()
        x, y = rot(a, b, p)
        assert x.requires_grad is a.requires_grad and y.requires_grad is b.requires_grad
        grad = x if a is q else y
        assert torch.autograd.grad(grad.sum(), q)[0].shape == q.shape
        assert calls[-1][1][13] == 2 and calls[-1][1][17] is None  # q's gradient alone is turned back
    # of a second derivative too
    x, y = rot(q, k, p)
    g, = torch.autograd.grad(x, q, torch.ones_like(x, requires_grad=True), create_graph=True)
    assert g.requires_grad and g.grad_fn is not None


def test_one_memory_is_not_turned_twice_at_once(calls):  # noqa: F811
    rot, p, x = mx.Rotary(32, device="cpu"), i32(0, 1, 2), torch.zeros(3, 2, 32)
    for k in (x, x[:, :1], x.detach()):
        with pytest.raises(ValueError, match="overlap"):
            rot(x, k, p, inplace=True)
    assert not calls and x._version == 0
    rot(x, x, p)
    rot(x[:, :1], x[:, 1:], p, inplace=True)
    rot(x[:0], x[:0], p[:0], inplace=True)
    assert len(calls) == 3


def test_results_that_ask_for_a_gradient_are_refused(calls):  # noqa: F811
    c = cache()
    table, cu = torch.zeros(1, 2, dtype=torch.int32), i32(0, 3)
    bf16 = lambda *s, grad=False: torch.zeros(*s, dtype=torch.bfloat16, requires_grad=grad)  # noqa: E731
    q, out, k, v = bf16(3, 4, 64), bf16(3, 4, 32, grad=True), bf16(3, 2, 64, grad=True), bf16(3, 2, 32, grad=True)
    for call in (lambda: c.attend(q, table, cu, out=out), lambda: c.read(table, cu, k_out=k, v_out=v.detach()),
                 lambda: c.read(table, cu, k_out=k.detach(), v_out=v)):
        with pytest.raises(ValueError, match="gradient"):
            call()
        assert not calls
        with torch.no_grad():
            call()
        calls.clear()
