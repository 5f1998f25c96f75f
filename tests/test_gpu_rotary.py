"""GPU parity of the rotary positions with the float64 oracle, forward and backward.

Tolerance: sine and cosine are off by 2^-22 at most (the fraction of a turn is formed in binary64 and used in two parts; the
functions themselves are good to a few units of 2^-24), the magnitude's product and the two products and their sum add
2^-24 of the magnitudes each: 2^-21 m (|a| + |b|) in all; then one rounding to the type."""

import math

import numpy as np
import pytest
import torch

import mixed_precision_moe_amd as mx
from mixed_precision_moe_amd import synth
from oracle import rotary as R

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
RAMP = dict(kind="ramp", factor=16.0, length=8192)


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def close(got, x, positions, rot, inverse=False):
    """got against the oracle's turn of x."""
    turns = rot._turns.cpu().numpy()
    x64 = x.detach().double().cpu().numpy()
    want = R.rotary_ref(x64, positions, turns, rot._offset, bool(rot._interleaved), rot._magnitude, inverse)
    mags = np.abs(x64).copy()
    n, o = len(turns), rot._offset
    a, b = (np.s_[..., o:o + 2 * n:2], np.s_[..., o + 1:o + 2 * n:2]) if rot._interleaved else (np.s_[..., o:o + n], np.s_[..., o + n:o + 2 * n])
    both = np.abs(x64[a]) + np.abs(x64[b])
    mags[a], mags[b] = both, both
    tol = 2.0 ** -21 * abs(rot._magnitude) * mags + HALF_STEP[x.dtype] * np.abs(want) + 1e-38
    rest = np.ones(x64.shape[-1], bool)
    rest[o:o + 2 * n] = False
    got64 = got.detach().double().cpu().numpy()
    assert np.array_equal(got64[..., rest], x64[..., rest])  # copied
    off = np.abs(got64 - want)
    assert np.all(off <= tol), float(np.max(off / tol))


def make(rows, heads, dim, dtype, seed=0):
    g = synth.rng(350, seed, rows, heads)
    return torch.from_numpy(g.standard_normal((rows, heads, dim)).astype(np.float32)).cuda().to(dtype)


def spread(rows, seed=1):
    g = np.random.default_rng(seed)
    p = g.integers(0, 1 << 20, rows)
    p[:3] = [0, 1, (1 << 31) - 1][:rows]
    if rows > 3:
        p[3] = -77
    return p


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,q_heads,k_heads,dim,rot,offset", [
    (1, 1, 1, 64, 64, 0), (1, 4, 2, 64, 64, 0), (7, 8, 2, 128, 128, 0), (33, 3, 1, 192, 64, 128), (5, 2, 2, 96, 32, 16),
    (4, 3, 1, 34, 34, 0), (3, 2, 1, 51, 6, 3), (9, 5, 5, 16, 2, 14), (2, 1, 1, 2, 2, 0), (3, 1, 1, 2050, 2048, 2), (6, 16, 4, 80, 40, 8)])
def test_both_directions(dtype, interleaved, rows, q_heads, k_heads, dim, rot, offset):
    print(f"rotary {dtype} rows={rows} heads={q_heads},{k_heads} dim={dim} rot={rot}+{offset} interleaved={interleaved}", flush=True)
    q, k, p = make(rows, q_heads, dim, dtype), make(rows, k_heads, dim, dtype, 1), spread(rows)
    r = mx.Rotary(rot, interleaved=interleaved, offset=offset, scaling=RAMP if rot > 2 else None)
    qo, ko = r(q.requires_grad_(), k.requires_grad_(), i32(p))
    close(qo, q, p, r)
    close(ko, k, p, r)
    gq, gk = make(rows, q_heads, dim, dtype, 2), make(rows, k_heads, dim, dtype, 3)
    dq, dk = torch.autograd.grad((qo, ko), (q, k), (gq, gk))
    close(dq, gq, p, r, True)
    close(dk, gk, p, r, True)


def test_angles_of_far_positions():
    """Positions near 2^31 and frequencies down to 10^-4: the fraction of a turn in exact arithmetic."""
    p = np.array([(1 << 31) - 1, -(1 << 31), 123456789, 99999999, 65537])
    for base in (10000.0, 5e5):
        r = mx.Rotary(64, base)
        x = torch.zeros(5, 1, 64, device="cuda")
        x[:, :, :32] = 1.0
        y, _ = r(x, None, i32(p))
        close(y, x, p, r)


def test_gradient_against_differences():
    """The sum of a weighting of the result, differentiated numerically (the operator is linear: one step is exact up to
    roundings of fp32, 2^-23 of the terms, over a step of 1)."""
    q, p = make(3, 2, 32, torch.float32), i32([5, 100, 7])
    w = make(3, 2, 32, torch.float32, 9)
    r = mx.Rotary(16, offset=8, interleaved=True, scaling=dict(kind="linear", factor=2.0))
    q.requires_grad_()
    (r(q, None, p)[0] * w).sum().backward()
    f = lambda x: float((r(x, None, p)[0].double() * w.double()).sum())  # noqa: E731
    base = q.detach()
    for at in [(0, 0, 0), (1, 1, 8), (2, 0, 9), (1, 0, 23), (2, 1, 31)]:
        step = base.clone()
        step[at] += 1.0
        assert f(step) - f(base) == pytest.approx(float(q.grad[at]), abs=2.0 ** -20 * 192)


def test_second_derivatives_and_one_gradient():
    q, k = make(4, 2, 32, torch.float32).requires_grad_(), make(4, 1, 32, torch.float32, 1).requires_grad_()
    p, r = i32([3, 2, 1, 0]), mx.Rotary(32)
    qo, ko = r(q, k, p)
    gk, = torch.autograd.grad(ko.sum(), k, retain_graph=True)  # expanded gradient, the queries without any
    close(gk, torch.ones_like(gk), [3, 2, 1, 0], r, True)
    gq, = torch.autograd.grad((qo ** 3).sum(), q, create_graph=True)
    h, = torch.autograd.grad(gq.sum(), q)
    # d/dq sum(R^T 3 (Rq)^2) = R^T (6 (Rq) * (R 1)), in float64
    turns = r._turns.cpu().numpy()
    x, one = q.detach().double().cpu().numpy(), np.ones((4, 2, 32))
    y, o = R.rotary_ref(x, [3, 2, 1, 0], turns), R.rotary_ref(one, [3, 2, 1, 0], turns)
    want = R.rotary_ref(6 * y * o, [3, 2, 1, 0], turns, inverse=True)
    assert np.all(np.abs(h.double().cpu().numpy() - want) <= 2.0 ** -18 * (np.abs(want) + 6 * np.abs(y).max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_slices_and_in_place(dtype, interleaved):
    """Queries and keys as views of one fused projection: turned beside it, and where they are."""
    p = [9, 0, 4000, 31, 8]
    for dim, pad in ((64, 8), (33, 1)):
        fused = make(5, 7, dim + pad, dtype)
        before = fused.clone()
        q, k = fused[:, :4, pad:], fused[:, 4:6, pad:]
        r = mx.Rotary(16, offset=dim - 16, interleaved=interleaved)
        qo, ko = r(q, k, i32(p))
        assert qo.is_contiguous() and torch.equal(fused, before)
        close(qo, q, p, r)
        close(ko, k, p, r)
        a, b = r(q, k, i32(p), inplace=True)
        assert a.data_ptr() == q.data_ptr() and torch.equal(a, qo) and torch.equal(b, ko)
        assert torch.equal(fused[:, 6], before[:, 6]) and torch.equal(fused[:, :, :pad], before[:, :, :pad])
        heads_first = make(7, 5, dim, dtype, 4).transpose(0, 1)  # heads outermost
        close(r(heads_first, None, i32(p))[0], heads_first, p, r)
    broadcast = make(5, 1, 64, dtype, 5).expand(5, 3, 64)
    close(r(broadcast[..., :dim], None, i32(p))[0], broadcast[..., :dim], p, r)


def test_gradients_of_broadcast_inputs():
    x = make(1, 1, 32, torch.float32).requires_grad_()
    p, r = [4, 7, 1000], mx.Rotary(32)
    y, _ = r(x.expand(3, 2, 32), None, i32(p))
    y.sum().backward()
    want = R.rotary_ref(np.ones((3, 2, 32)), p, r._turns.cpu().numpy(), inverse=True).sum((0, 1))
    assert np.all(np.abs(x.grad.double().cpu().numpy()[0, 0] - want) <= 6 * 2.0 ** -20)


def test_nothing_to_do_and_values_that_are_not_numbers():
    r = mx.Rotary(32)
    z = torch.zeros(0, 2, 32, dtype=torch.bfloat16, device="cuda")
    q, k = r(z, z[:, :1], i32([]))
    assert q.shape == (0, 2, 32) and k.shape == (0, 1, 32)
    x = make(4, 2, 32, torch.bfloat16)
    want = r(x, None, i32([1, 2, 3, 4]))[0]
    x[1, 1, 3] = float("nan")
    y = r(x, None, i32([1, 2, 3, 4]))[0]
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1, 1, [3, 19]] = True
    assert bool(torch.isnan(y[bad]).all()) and torch.equal(y[~bad], want[~bad])


def test_many_rows():
    """More groups of rows than workgroups."""
    n = (1 << 20) * 4 + 5
    x = torch.ones(n, 1, 2, device="cuda", dtype=torch.bfloat16)
    r = mx.Rotary(2, freqs=[2 * math.pi / 4])  # a quarter turn a position
    y = r(x, None, torch.arange(n, device="cuda").int())[0][:, 0]
    a, b = x[0, 0]
    for k, want in enumerate(((a, b), (-b, a), (-a, -b), (b, -a))):
        assert torch.equal(y[k::4], torch.stack(want).expand_as(y[k::4]))


def test_streams_graphs_and_other_devices(monkeypatch):
    q, k = make(9, 4, 64, torch.bfloat16), make(9, 2, 64, torch.bfloat16, 1)
    p, r = i32(list(range(9))), mx.Rotary(64, scaling=RAMP)
    want = r(q, k, p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = r(q, k, p)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = r(q, k, p)
    for i in range(4):
        q.copy_(make(9, 4, 64, torch.bfloat16, 10 + i))
        p.copy_(i32([1000 * i + x for x in range(9)]))
        graph.replay()
        torch.cuda.synchronize()
        eager = r(q, k, p)
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
        close(out[0], q, p.tolist(), r)
    monkeypatch.setattr(mx.ops, "_current_gpu", lambda: -1)  # as if another device were the current one
    assert torch.equal(r(q, k, p)[0], eager[0])


def test_a_captured_training_pass():
    x = make(6, 2, 32, torch.float32).requires_grad_()
    p, r = i32([5, 4, 3, 2, 1, 0]), mx.Rotary(32)
    g = make(6, 2, 32, torch.float32, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # a first pass, whose graph ends here
        torch.autograd.grad(r(x, None, p)[0], x, g)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = r(x, None, p)[0]
        dx, = torch.autograd.grad(y, x, g)
        y = y.detach()
    for i in range(4):
        with torch.no_grad():
            x.copy_(make(6, 2, 32, torch.float32, 20 + i))
        p.copy_(i32([7 * i + j for j in range(6)]))
        graph.replay()
        torch.cuda.synchronize()
        close(y, x, p.tolist(), r)
        close(dx, g, p.tolist(), r, True)


def test_refusals():
    r = mx.Rotary(32)
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    q, k, p = z(3, 2, 32), z(3, 1, 32), i32([0, 1, 2])
    bad = [lambda: r(q.half(), k.half(), p), lambda: r(q, k.float(), p), lambda: r(q, k[:2], p), lambda: r(q, z(3, 1, 64), p),
           lambda: r(q, k, p.long()), lambda: r(q, k, p[:2]), lambda: r(q, k, i32([0, 0, 0, 0, 0, 0])[::2]), lambda: r(q.cpu(), k, p),
           lambda: r(q, k, p.cpu()), lambda: r(z(3, 2, 16), None, p), lambda: r(z(3, 32, 2).transpose(1, 2), None, p),
           lambda: r(z(3, 0, 32), None, p), lambda: r(q[0], None, p), lambda: r(q.clone().requires_grad_(), None, p, inplace=True)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(mx.Mxfp4Error):  # results on each other
        r(z(1, 1, 32).expand(3, 2, 32), None, p, inplace=True)
