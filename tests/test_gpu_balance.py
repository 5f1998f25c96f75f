"""GPU parity of the balance loss, its counts and its gradient with the float64 oracle.

Tolerances, from the arithmetic (u = 2^-24, one binary32 rounding).  A probability exp(l - m) / s: l - m and its
product with log2(e) are rounded, which moves the exponential by at most R u each, R the row's range; the
exponential, the sum over the row (at most 24 additions in sequence) and the division add 30 u: dp = (2 R + 30) u of
itself.  The loss is an average of probabilities with weights >= 0: dp, plus the additions of a lane's rows and of
the workgroup's partial sums (at most 64 + T / 2048 in sequence), plus its own rounding.  The gradient
g p (d - mean): the bracket's terms are at most 2 D with D = max |d|, the second mean leaves of the first one's
rounding only its product with the error of sum p, so the bracket is off by at most 2 D (dp + 32 u).
"""

import numpy as np
import pytest
import torch

import mixed_precision_moe_amd as mx
from mixed_precision_moe_amd import synth
from oracle import balance as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def case(T, E, k, seed, mask=False, spread=1.5):
    g = synth.rng(300, seed, T, E, k)
    l = (g.standard_normal((T, E)) + spread * g.standard_normal((1, E))).astype(np.float32)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    return l, ids, (g.random(T) < 0.7) if mask else None


def device_inputs(l, ids, mask):
    return (torch.from_numpy(l).cuda().requires_grad_(), torch.from_numpy(np.ascontiguousarray(ids)).cuda(),
            None if mask is None else torch.from_numpy(mask).cuda())


def assert_close(loss, counts, grad, l, ids, mask, w):
    ref, n, gref = B.balance_ref(l, ids, mask, float(np.float32(w)))
    T, E = l.shape
    np.testing.assert_array_equal(counts.cpu().numpy(), n)
    fin = np.where(np.isfinite(l), l, np.nan)
    live = np.arange(T) if mask is None else np.flatnonzero(mask)
    R = 0.0
    if live.size:
        with np.errstate(all="ignore"):
            R = float(np.nanmax(np.nan_to_num(np.nanmax(fin[live], 1) - np.nanmin(fin[live], 1))))
    dp = (2 * R + 30) * U
    assert abs(loss.item() - ref) <= ref * (dp + (66 + T / 2048) * U)
    got = grad.cpu().numpy().astype(np.float64)
    V, k = max(1, live.size), ids.shape[1]
    D = E / (k * V ** 2) * np.abs(n - n.mean()).max()
    p = np.zeros((T, E))
    if live.size:
        p[live] = B.softmax_rows(l[live])
    # 2^-149: the smallest step of binary32
    bound = abs(float(np.float32(w))) * p * 2 * D * (dp + 32 * U) + 2 * dp * np.abs(gref) + 2.0 ** -149
    assert np.all(np.abs(got - gref) <= bound)
    if mask is not None:
        assert not got[~mask].any()


def run(l, ids, mask, w=0.01):
    ld, idd, md = device_inputs(l, ids, mask)
    loss, counts = mx.balance_loss(ld, idd, md)
    grad, = torch.autograd.grad(loss, ld, torch.tensor(w, device="cuda"))
    return loss, counts, grad


# experts on both sides of every row shape, divisible by four (vector loads) and not; one workgroup and many
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 1), (16, 4, 2), (3, 16, 4), (700, 17, 3), (129, 32, 8), (513, 33, 5),
                                   (65, 64, 6), (300, 65, 2), (64, 128, 8), (4099, 128, 8), (77, 130, 4), (50, 256, 8),
                                   (33, 257, 1), (1000, 384, 8), (21, 385, 32), (40, 512, 8), (19, 513, 7),
                                   (300, 768, 8), (9, 769, 2), (200, 1024, 8), (7, 1021, 3)])
@pytest.mark.parametrize("masked", [False, True])
def test_shapes(T, E, k, masked):
    print(f"balance T={T} E={E} k={k} masked={masked}", flush=True)
    l, ids, mask = case(T, E, k, 1, masked)
    loss, counts, grad = run(l, ids, mask)
    assert_close(loss, counts, grad, l, ids, mask, 0.01)
    # the same bits again
    loss2, counts2, grad2 = run(l, ids, mask)
    assert torch.equal(loss, loss2) and torch.equal(counts, counts2) and torch.equal(grad, grad2)


def test_many_tokens():
    l, ids, mask = case(40001, 60, 4, 2, True)
    assert_close(*run(l, ids, mask, -3.0), l, ids, mask, -3.0)


def test_no_tokens_and_masks_that_leave_nothing():
    l, ids, _ = case(50, 12, 3, 3)
    for T, mask in ((0, None), (50, np.zeros(50, bool)), (0, np.zeros(0, bool))):
        loss, counts, grad = run(l[:T], ids[:T], mask)
        assert loss.item() == 0.0 and not counts.any() and not grad.any() and grad.shape == (T, 12)
    l, ids, _ = case(3000, 96, 3, 3)  # several workgroups
    loss, counts, grad = run(l, ids, np.zeros(3000, bool))
    assert loss.item() == 0.0 and not counts.any() and not grad.any()


@pytest.mark.parametrize("T", [40, 3000])
def test_masked_tokens_may_hold_anything(T):
    l, ids, mask = case(T, 48, 4, 4, True)
    clean = run(l, ids, mask)
    l2, ids2 = l.copy(), ids.copy()
    dead = np.flatnonzero(~mask)
    l2[dead] = np.array([np.nan, np.inf, -np.inf, 3e38], np.float32)[np.arange(dead.size) % 4][:, None]
    ids2[dead] = np.iinfo(np.int32).max
    for a, b in zip(clean, run(l2, ids2, mask)):
        assert torch.equal(a, b)


def test_excluded_experts_and_rows_without_any():
    """Logits of -inf have no probability; a row of them has none at all and no gradient.  The type's lowest finite
    value is a logit like any other."""
    l, ids, _ = case(200, 20, 2, 5)
    l[:, 7] = -np.inf
    l[3] = -np.inf
    l[4, 5:] = np.finfo(np.float32).min
    l[5] = np.finfo(np.float32).min
    loss, counts, grad = run(l, ids, None, 1.0)
    ref, n, gref = B.balance_ref(l, ids)
    np.testing.assert_array_equal(counts.cpu().numpy(), n)
    # the finite rows' ranges: row 4's probabilities are exact zeros past column 5
    R = float(np.nanmax(np.where(np.isfinite(l) & (l > -1e30), l, np.nan)) - np.nanmin(np.where(np.isfinite(l) & (l > -1e30), l, np.nan)))
    dp = (2 * R + 30) * U
    assert abs(loss.item() - ref) <= ref * (dp + 67 * U)
    got = grad.cpu().numpy()
    assert np.all(np.isfinite(got)) and not got[3].any() and not got[~np.isfinite(l)].any()
    D = 20 / (2 * 200 ** 2) * np.abs(n - n.mean()).max()
    assert np.all(np.abs(got - gref) <= B.softmax_rows(l) * 2 * D * (dp + 32 * U) + 2 * dp * np.abs(gref) + 2.0 ** -149)


@pytest.mark.parametrize("T,E", [(30, 24), (900, 27)])
def test_dropped_pairs(T, E):
    l, ids, mask = case(T, E, 4, 6, True)
    ids[::3, 1] = -1
    ids[1::5, 3] = E
    ids[2::7] = np.iinfo(np.int32).min
    assert_close(*run(l, ids, mask), l, ids, mask, 0.01)


def test_the_same_expert_twice_and_one_expert_for_all():
    l, ids, _ = case(500, 16, 4, 7)
    ids[:] = 5
    assert_close(*run(l, ids, None), l, ids, None, 0.01)


def test_peaked_rows_keep_their_small_gradients():
    """One expert holds nearly all of each row: the gradient is p (1 - p) sized and the bracket cancels."""
    l, ids, _ = case(64, 8, 2, 8)
    l[np.arange(64), ids[:, 0]] += 12.0
    loss, counts, grad = run(l, ids, None, 1.0)
    _, _, gref = B.balance_ref(l, ids)
    R = float((l.max(1) - l.min(1)).max())
    # relative to the whole gradient, not to D: what is left of the bracket is sum over the others of p (d - d_top)
    err = np.abs(grad.cpu().numpy() - gref)
    assert err.max() <= np.abs(gref).max() * (4 * R + 100) * U


@pytest.mark.parametrize("T,E,off,pad", [(70, 32, 0, 5), (70, 32, 1, 8), (600, 64, 3, 1), (600, 64, 0, 4)])
def test_strided_and_misaligned_rows(T, E, off, pad):
    l, ids, mask = case(T, E, 3, 9, True)
    buf = torch.full((T, off + E + pad), float("nan"), device="cuda")
    buf[:, off:off + E] = torch.from_numpy(l).cuda()
    view = buf[:, off:off + E].detach().requires_grad_()
    loss, counts = mx.balance_loss(view, torch.from_numpy(ids).cuda(), torch.from_numpy(mask).cuda().to(torch.uint8) * 255)
    grad, = torch.autograd.grad(loss, view, torch.tensor(0.01, device="cuda"))
    assert_close(loss, counts, grad, l, ids, mask, 0.01)


@pytest.mark.parametrize("T,E,off,pad", [(8, 4, 0, 12), (70, 32, 1, 8), (600, 64, 0, 64)])
def test_strided_rows_under_saved_tensor_hooks(T, E, off, pad):
    """The rows come back from the host without the space between them."""
    l, ids, mask = case(T, E, 3, 9, True)
    buf = torch.full((T, off + E + pad), float("nan"), device="cuda")
    buf[:, off:off + E] = torch.from_numpy(l).cuda()
    view = buf[:, off:off + E].detach().requires_grad_()
    with torch.autograd.graph.save_on_cpu():
        loss, counts = mx.balance_loss(view, torch.from_numpy(ids).cuda(), torch.from_numpy(mask).cuda())
    grad, = torch.autograd.grad(loss, view, torch.tensor(0.01, device="cuda"))
    assert_close(loss, counts, grad, l, ids, mask, 0.01)


def test_gradient_against_differences():
    """Central differences of the device's own loss, h = 2^-5: the curvature term h^2/6 |f'''| is below 2^-10 of the
    bound p D on the gradient, the loss's rounding 2^-24 f / h is the other allowance."""
    l, ids, _ = case(6, 5, 2, 10)
    _, _, grad = run(l, ids, None, 1.0)
    h = 2.0 ** -5
    for t in range(6):
        for e in range(5):
            f = []
            for s in (h, -h):
                m = l.copy()
                m[t, e] += s
                f.append(run(m, ids, None)[0].item())
            step = float(np.float32(l[t, e] + np.float32(h))) - float(np.float32(l[t, e] - np.float32(h)))
            _, n, _ = B.balance_ref(l, ids)
            D = 5 / (2 * 36) * np.abs(n - n.mean()).max()
            assert abs((f[0] - f[1]) / step - float(grad[t, e])) <= 2.0 ** -10 * D + 40 * U * max(f) / step * 2


def test_in_a_training_step():
    """The loss added to another one: gradients accumulate in the leaf, upstream weights reach it, and a second
    backward is refused as for any node whose tensors were freed."""
    l, ids, _ = case(90, 12, 2, 11)
    base = torch.from_numpy(l).cuda()
    idd = torch.from_numpy(ids).cuda()
    w = torch.ones(12, device="cuda", requires_grad=True)
    loss, counts = mx.balance_loss(base * w, idd)
    assert not counts.requires_grad and loss.shape == ()
    total = 0.3 * loss + (w * w).sum()
    total.backward()
    _, _, gref = B.balance_ref(l, ids, None, float(np.float32(0.3)))
    want = (gref * l).sum(0) + 2.0
    # as the gradient's tolerance above, summed over the column's 90 products
    D = 12 / (2 * 90 ** 2) * 90
    tol = (0.3 * np.abs(l).sum(0) * 2 * D * 2 ** -18 + np.abs(gref * l).sum(0) * 2 ** -16 + 2 * 2 ** -22)
    assert np.all(np.abs(w.grad.cpu().numpy() - want) <= tol)
    with pytest.raises(RuntimeError):
        loss.backward()
    with torch.no_grad():
        assert not mx.balance_loss(base, idd)[0].requires_grad
    loss, counts = mx.balance_loss(base.requires_grad_(), idd)  # only the counts are used
    assert counts.sum().item() == 180


def test_very_many_tokens():
    l, ids, mask = case(300007, 8, 2, 15, True)
    assert_close(*run(l, ids, mask), l, ids, mask, 0.01)


def test_second_derivatives_and_changed_logits_are_refused():
    l, ids, _ = case(20, 6, 2, 16)
    ld, idd, _ = device_inputs(l, ids, None)
    loss, _ = mx.balance_loss(ld, idd)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(loss, ld, create_graph=True)
    x = ld * 1.0
    loss, _ = mx.balance_loss(x, idd)
    x.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_calls_on_two_streams_at_once_and_from_another_device(monkeypatch):
    l, ids, mask = case(5000, 96, 4, 17, True)
    ld, idd, md = device_inputs(l, ids, mask)
    want = [t.detach().clone() for t in run(l, ids, mask, 0.5)]
    w = torch.tensor(0.5, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            loss, counts = mx.balance_loss(ld, idd, md)
            got.append((loss, counts, torch.autograd.grad(loss, ld, w)[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    monkeypatch.setattr(mx.ops, "_current_gpu", lambda: -1)  # as if another device were the current one
    assert all(torch.equal(a, b) for a, b in zip(run(l, ids, mask, 0.5), want))


def test_on_another_stream_and_in_a_graph():
    l, ids, mask = case(2000, 128, 8, 12, True)
    ld, idd, md = device_inputs(l, ids, mask)
    w = torch.tensor(0.5, device="cuda")

    def step():
        loss, counts = mx.balance_loss(ld, idd, md)
        return loss, counts, torch.autograd.grad(loss, ld, w)[0]

    want = [t.detach().clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del got  # no eager graph of these leaves lives while their backward is captured
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    other = torch.from_numpy(case(2000, 128, 8, 13)[0]).cuda()
    for i in range(4):
        with torch.no_grad():
            ld.copy_(other if i % 2 else torch.from_numpy(l).cuda())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.detach().clone() for t in out]
        eager = [t.detach().clone() for t in step()]
        assert all(torch.equal(a, b) for a, b in zip(got, eager))
        if i % 2 == 0:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    l, ids, _ = case(8, 6, 2, 14)
    l, ids = torch.from_numpy(l).cuda(), torch.from_numpy(ids).cuda()
    for bad in (lambda: mx.balance_loss(l.half(), ids), lambda: mx.balance_loss(l[0], ids),
                lambda: mx.balance_loss(l, ids.long()), lambda: mx.balance_loss(l, ids[:7]),
                lambda: mx.balance_loss(l, ids.t().contiguous().t()), lambda: mx.balance_loss(l.t().contiguous().t(), ids),
                lambda: mx.balance_loss(l[:1].expand(8, 6), ids),
                lambda: mx.balance_loss(l, ids.cpu()), lambda: mx.balance_loss(l, ids, torch.ones(7, device="cuda") > 0),
                lambda: mx.balance_loss(l, ids, torch.ones(8, device="cuda")),
                lambda: mx.balance_loss(l, ids, torch.ones(8) > 0),
                lambda: mx.balance_loss(torch.zeros(4, 1025, device="cuda"), ids[:4])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(mx.Mxfp4Error):  # more pairs a token than experts
        mx.balance_loss(l, ids.repeat(1, 4))
