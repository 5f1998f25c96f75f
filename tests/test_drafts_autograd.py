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
