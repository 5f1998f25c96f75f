"""GPU parity of the 4-bit matrix-vector products, dense and per routed pair, with the float64 oracle.

Tolerance, from the arithmetic (u = 2^-24).  Weights times their scales are exact in bf16 and so are the products
in binary32; an output is a sum of K products, of which at most 32 inside one matrix instruction, then K / 128
accumulations in sequence and 16 partial sums add a rounding each (counted twice, whichever way the matrix unit
rounds): 2 (K / 128 + 48) u of sum |x W|.  (Few rows of x with NVFP4 weights: two matrix instructions sum a block of 16, and
2 K / 128 multiply-adds with its scale follow, one rounding each: the same bound.)  The global scale's division and the bias add 2 u each of what they give, and
the result is rounded once: 2^-9 of itself to bf16 and half an ulp (2^-8 bounds it at every place of a binade) or u.
SwiGLU: silu has a slope of at most 1.1, its own evaluation errs by (|g| + 8) u.
"""

import numpy as np
import pytest
import torch

import mixed_precision_moe_amd as mx
from mixed_precision_moe_amd import synth
from oracle import matvec as V
from oracle import quant as Q
from tests.gpu_common import bf16_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
FMTS = {"mxfp4": mx.FMT_MXFP4, "nvfp4": mx.FMT_NVFP4}


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def weights(g, shape, fmt, sigma=0.02):
    """Quantized weights [..., N, K]: (q, s, global scale or None) on the host."""
    N, K = shape[-2:]
    gs = float(np.float32(448.0 / sigma)) if fmt == "nvfp4" else None
    q, s = [], []
    for _ in range(int(np.prod(shape[:-2]))):
        w = synth.to_bf16_bits(g.standard_normal((N, K), dtype=np.float32) * np.float32(sigma))
        a, b = Q.nvfp4_quantize_ref(w, gs) if fmt == "nvfp4" else Q.quantize_ref(w)
        q.append(a)
        s.append(b)
    return np.stack(q).reshape(*shape[:-1], -1), np.stack(s).reshape(*shape[:-1], -1), gs


def linear_bound(y, mag, K, b=None):
    base = mag if b is None else mag + np.abs(b)
    return 2 * (K / 128 + 48) * U * mag + 4 * U * base


def assert_dense(y, x_bits, q, s, gs, b, out):
    ref, mag = V.matvec_ref(x_bits, q, s, b, gs)
    K = x_bits.shape[1]
    err = np.abs(host(y) - ref)
    bound = linear_bound(ref, mag, K, b) + (2.0 ** -8 if out == torch.bfloat16 else U) * np.abs(ref) + 2.0 ** -133
    assert y.shape == ref.shape and np.all(err <= bound), float((err / bound).max())


def dense(M, N, K, fmt, bias, out=torch.bfloat16, pad=0, seed=0):
    print(f"matvec {fmt} M={M} N={N} K={K} bias={bias} out={out} pad={pad}", flush=True)
    g = synth.rng(310, seed, M, N, K)
    q, s, gs = weights(g, (N, K), fmt)
    x = synth.to_bf16_bits(g.standard_normal((M, K), dtype=np.float32))
    bt, b = None, None
    if bias:
        bt = torch.from_numpy(g.normal(0, 0.5, N).astype(np.float32)).cuda()
        bt = bt.bfloat16() if bias == "bf16" else bt
        b = host(bt)
    buf = np.full((M, K + pad), 0x7FC0, np.uint16)  # NaN between the rows
    buf[:, :K] = x
    xd = bf16_dev(buf)[:, :K]
    qd, sd = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    y = mx.fp4_matvec(xd, qd, sd, bt, fmt=FMTS[fmt], global_scale=gs, out_dtype=out)
    assert y.dtype == out
    assert_dense(y, x, q, s, gs, b, out)
    assert torch.equal(y, mx.fp4_matvec(xd, qd, sd, bt, fmt=FMTS[fmt], global_scale=gs, out_dtype=out))
    return xd, qd, sd, gs, y


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("M", [1, 4, 8, 16])
def test_large_and_small_rows_scale_exactly(fmt, M):
    """A power of two on x is one on y: nothing on the way overflows or goes below binary32's normal range."""
    xd, qd, sd, gs, y = dense(M, 37, 1040 if fmt == "nvfp4" else 1056, fmt, None, torch.float32, seed=5)
    for e in (100, -90):
        z = mx.fp4_matvec((xd.float() * 2.0 ** e).bfloat16(), qd, sd, fmt=FMTS[fmt], global_scale=gs, out_dtype=torch.float32)
        assert torch.equal(z.double(), y.double() * 2.0 ** e)


# rows below, at and past a tile of 16; outputs that fill no tile; K of one block, below a step, ragged, long
@pytest.mark.parametrize("fmt,M,N,K,bias", [
    ("mxfp4", 1, 1, 32, None), ("mxfp4", 1, 16, 32, "bf16"), ("mxfp4", 2, 17, 96, "fp32"), ("mxfp4", 1, 256, 256, "bf16"),
    ("mxfp4", 16, 33, 128, None), ("mxfp4", 17, 40, 160, "fp32"), ("mxfp4", 5, 64, 1056, None), ("mxfp4", 3, 48, 7168, None),
    ("mxfp4", 33, 100, 2048, "bf16"), ("mxfp4", 70, 31, 544, None), ("mxfp4", 4, 20, 8192, None), ("mxfp4", 4, 33, 16416, None),
    ("mxfp4", 9, 17, 20000, "fp32"), ("nvfp4", 3, 18, 8208, None), ("nvfp4", 4, 16, 24592, None), ("nvfp4", 16, 16, 16368, None),
    ("nvfp4", 1, 1, 32, None), ("nvfp4", 1, 5, 48, "fp32"), ("nvfp4", 4, 16, 112, None), ("nvfp4", 16, 65, 128, "bf16"),
    ("nvfp4", 21, 99, 2032, "bf16"), ("nvfp4", 2, 48, 7168, None), ("nvfp4", 8, 50, 1040, "fp32"), ("nvfp4", 34, 20, 272, None)])
def test_shapes(fmt, M, N, K, bias):
    dense(M, N, K, fmt, bias)


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 9, 16, 32])
def test_fp32_output_and_padded_rows(fmt, M):
    dense(M, 70, 384, fmt, "fp32", torch.float32, pad=40, seed=1)


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("M", [3, 4, 7, 16, 40])
def test_rows_that_are_not_finite_stay_among_themselves(fmt, M):
    xd, qd, sd, gs, y = dense(M, 130, 1088, fmt, None, torch.float32, seed=2)
    bad = xd.clone()
    bad[1] = float("nan")
    bad[M - 1] = float("inf")
    z = mx.fp4_matvec(bad, qd, sd, fmt=FMTS[fmt], global_scale=gs, out_dtype=torch.float32)
    keep = [i for i in range(M) if i not in (1, M - 1)]
    assert torch.equal(z[keep], y[keep]) and not torch.isfinite(z[1]).any() and not torch.isfinite(z[M - 1]).any()


def loud_neighbours(shape, fmt):
    """Weights whose odd rows are the largest the contract allows (MXFP4: 2^127) or NaN (NVFP4), and the same with odd
    rows of zeros.  K ends inside a step, so a row's last step lies beside the next row's scales."""
    g = synth.rng(316, *shape)
    *rows, K = shape
    q = g.integers(0, 256, (*rows, K // 2), dtype=np.uint8)
    q[..., ::2, -8:] = 0x7F  # 6 and -6 where a scale that is not the row's own would overflow them
    if fmt == "mxfp4":
        s = np.full((*rows, K // 32), 120, np.uint8)
        s[..., 1::2, :] = 254
        q[..., 1::2, :] = 0x22  # ones
    else:
        s = np.full((*rows, K // 16), 0x38, np.uint8)
        s[..., 1::2, :] = 0x7F
    quiet_q, quiet_s = q.copy(), s.copy()
    quiet_q[..., 1::2, :] = 0
    quiet_s[..., 1::2, :] = 0
    return [torch.from_numpy(t).cuda() for t in (q, s, quiet_q, quiet_s)]


@pytest.mark.parametrize("fmt,K", [("mxfp4", 32), ("mxfp4", 96), ("mxfp4", 1056), ("nvfp4", 32), ("nvfp4", 48), ("nvfp4", 112),
                                   ("nvfp4", 1040)])
@pytest.mark.parametrize("M", [1, 3, 8, 16])
def test_a_rows_scales_touch_no_other_row(fmt, K, M):
    q, s, quiet_q, quiet_s = loud_neighbours((39, K), fmt)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(K)).bfloat16().cuda()
    gs = {"fmt": FMTS[fmt], "global_scale": 1.0 if fmt == "nvfp4" else None, "out_dtype": torch.float32}
    y, z = mx.fp4_matvec(x, q, s, **gs), mx.fp4_matvec(x, quiet_q, quiet_s, **gs)
    assert torch.isfinite(z).all() and torch.equal(y[:, ::2], z[:, ::2])


# the second shape has four tiles a wave
@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("E,N,K,pairs", [(6, 39, 1056, 3), (6, 39, 1056, 9), (64, 1024, 1568, 4), (64, 1024, 1568, 11)])
def test_an_experts_scales_touch_no_other_row(fmt, E, N, K, pairs):
    q, s, quiet_q, quiet_s = loud_neighbours((E, N, K), fmt)
    P = pairs * E
    x = torch.randn(P, K, generator=torch.Generator().manual_seed(K)).bfloat16().cuda()
    offs = torch.arange(0, P + 1, pairs, dtype=torch.int32, device="cuda")
    listed = torch.arange(P, dtype=torch.int32, device="cuda")
    kw = {"fmt": FMTS[fmt], "global_scales": torch.ones(E, device="cuda") if fmt == "nvfp4" else None, "out_dtype": torch.float32}
    y, z = mx.fp4_expert_matvec(x, q, s, offs, listed, **kw), mx.fp4_expert_matvec(x, quiet_q, quiet_s, offs, listed, **kw)
    assert torch.isfinite(z).all() and torch.equal(y[:, ::2], z[:, ::2])


def test_every_code_and_scale():
    """Each E2M1 code under scales over the formats' normal ranges, one at a time against a unit vector: exact."""
    K, N = 64, 120
    g = synth.rng(311)
    x = np.zeros((16, K), np.uint16)
    x[np.arange(16), np.arange(0, 64, 4)] = 0x3F80
    q = g.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = g.integers(3, 252, (N, 2), dtype=np.uint8)  # 0.5 * 2^-124 .. 6 * 2^124
    y = mx.fp4_matvec(bf16_dev(x), torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), out_dtype=torch.float32)
    np.testing.assert_array_equal(host(y), V.matvec_ref(x, q, s)[0])
    s = np.arange(N * 4, dtype=np.uint16).reshape(N, 4) % 127  # every finite, non-negative E4M3 value
    s = s.astype(np.uint8)
    y = mx.fp4_matvec(bf16_dev(x), torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), fmt=mx.FMT_NVFP4, global_scale=1.0,
                      out_dtype=torch.float32)
    np.testing.assert_array_equal(host(y), V.matvec_ref(x, q, s, None, 1.0)[0])


@pytest.mark.parametrize("k", [-140, -120, 100, 127])
def test_extreme_global_scales(k):
    """A power of two as global scale moves the exponent and nothing else: also one whose reciprocal overflows, or has
    no full precision."""
    g = synth.rng(316)
    q = g.integers(0, 256, (40, 48), dtype=np.uint8)
    s = g.integers(1, 127, (40, 6), dtype=np.uint8)
    e = 40 if k > 0 else -60  # keeps the quotients in range
    x = synth.to_bf16_bits(g.standard_normal((2, 96)) * 2.0 ** e)
    args = (bf16_dev(x), torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda())
    one = host(mx.fp4_matvec(*args, fmt=mx.FMT_NVFP4, global_scale=1.0, out_dtype=torch.float32))
    y = host(mx.fp4_matvec(*args, fmt=mx.FMT_NVFP4, global_scale=2.0 ** k, out_dtype=torch.float32))
    want = np.ldexp(one, -k)
    keep = np.abs(want) >= 2.0 ** -126
    assert keep.any()
    np.testing.assert_array_equal(y[keep], want[keep])


def test_equals_the_linear_layer():
    """Against mx.Linear on the same weights, within both layers' tolerances."""
    g = synth.rng(312)
    w = synth.to_bf16_bits(g.standard_normal((192, 256), dtype=np.float32) * np.float32(0.02))
    q, s, _ = mx.quantize(bf16_dev(w), flat=True, tiled=False)
    x = synth.to_bf16_bits(g.standard_normal((7, 256), dtype=np.float32))
    a, b = host(mx.Linear(q, s)(bf16_dev(x))), host(mx.fp4_matvec(bf16_dev(x), q, s))
    rms = np.sqrt(np.mean(b ** 2))
    assert np.abs(a - b).max() <= 2e-2 * rms + 1e-3 + 2.0 ** -8 * np.abs(b).max()


def pairs_of(ids, E):
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    offs = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    return torch.from_numpy(offs.astype(np.int32)).cuda(), torch.from_numpy(order.astype(np.int32)).cuda()


def expert(T, E, k, N, K, fmt, swiglu, shared, bias, out=torch.bfloat16, seed=0, crowd=False):
    print(f"expert {fmt} T={T} E={E} k={k} N={N} K={K} swiglu={swiglu} shared={shared} bias={bias}", flush=True)
    g = synth.rng(313, seed, T, E, N)
    q, s, gs = weights(g, (E, N, K), fmt)
    gsv = None if gs is None else (gs * (0.5 + np.arange(E) / E)).astype(np.float32)
    x = synth.to_bf16_bits(g.standard_normal((T if shared else T * k, K), dtype=np.float32))
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    if crowd:
        ids[:] = ids[0]
    b = g.normal(0, 0.1, (E, N)).astype(np.float32) if bias else None
    offs, sp = pairs_of(ids, E)
    args = (bf16_dev(x), torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), offs, sp,
            None if b is None else torch.from_numpy(b).cuda())
    kw = dict(fmt=FMTS[fmt], global_scales=None if gsv is None else torch.from_numpy(gsv).cuda(), top_k=k if shared else 1,
              swiglu=swiglu, out_dtype=out)
    y = mx.fp4_expert_matvec(*args, **kw)
    h, mag = V.expert_matvec_ref(x, q, s, ids, shared, b, gsv)
    tol = linear_bound(h, mag, K, None if b is None else b[ids.reshape(-1)])
    ref = h
    if swiglu:
        ref = V.swiglu_ref(h)
        gate, up = np.split(h, 2, 1)
        tg, tu = np.split(tol, 2, 1)
        silu = gate / (1 + np.exp(-gate))
        tol = 1.1 * tg * (np.abs(up) + tu) + np.abs(silu) * tu + (np.abs(gate) + 8) * U * np.abs(ref)
    tol = tol + (2.0 ** -8 if out == torch.bfloat16 else U) * np.abs(ref) + 2.0 ** -133
    err = np.abs(host(y) - ref)
    assert y.shape == ref.shape and y.dtype == out and np.all(err <= tol), float((err / tol).max())
    assert torch.equal(y, mx.fp4_expert_matvec(*args, **kw))
    return args, kw, y


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("T,E,k,N,K,swiglu,shared,bias", [
    (1, 1, 1, 16, 32, False, True, False), (1, 8, 3, 34, 96, True, True, True), (5, 4, 2, 50, 160, False, False, True),
    (16, 70, 4, 32, 64, True, True, False), (33, 5, 5, 30, 224, True, False, True), (3, 200, 8, 18, 544, False, True, False)])
def test_experts(fmt, T, E, k, N, K, swiglu, shared, bias):
    expert(T, E, k, N, K, fmt, swiglu, shared, bias)


# blocks of four steps, with one to four rows an expert, more than a tile, and sixteen waves
@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("T,E,k,N,K,swiglu,shared,bias", [
    (1, 6, 1, 34, 512, True, True, True), (1, 6, 2, 34, 8224, True, True, False), (2, 5, 2, 20, 8224, False, False, True),
    (7, 6, 3, 40, 2048, True, True, True), (9, 20, 4, 33, 1056, False, True, True), (45, 5, 2, 38, 1024, True, False, True)])
def test_experts_with_long_rows(fmt, T, E, k, N, K, swiglu, shared, bias):
    expert(T, E, k, N, K, fmt, swiglu, shared, bias, torch.float32 if T == 1 else torch.bfloat16)


# pairs of the experts in turn: mostly up to 4, mostly 5 to 8, up to more than two tiles of x; none among them
PAIRS = {4: (4, 1, 3, 4, 0, 2, 4, 5, 4, 3), 8: (5, 8, 0, 6, 1, 7, 4), 16: (9, 16, 3, 12, 17, 0, 8, 33, 5)}


# Four tiles of 16 rows a wave: experts with three pairs on average or more, K of 1536 or more and 4096 tiles in all.
# Outputs end in the first, second and third of a workgroup's tiles, inside a tile and at its end; K ends inside a step.
@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("E,n_out,K,most,swiglu,bias,out", [
    (1010, 65, 1568, 4, False, None, torch.float32), (1010, 65, 1536, 4, True, "fp32", torch.bfloat16),
    (820, 80, 1808, 8, False, "bf16", torch.bfloat16), (600, 100, 1584, 8, True, None, torch.float32),
    (512, 128, 2048, 16, False, "fp32", torch.float32), (300, 219, 1552, 16, True, "bf16", torch.bfloat16)])
def test_four_tiles_a_wave(fmt, E, n_out, K, most, swiglu, bias, out):
    if fmt == "mxfp4":
        K = -(-K // 32) * 32
    print(f"four tiles {fmt} E={E} n_out={n_out} K={K} most={most} swiglu={swiglu} bias={bias}", flush=True)
    counts = np.resize(PAIRS[most], E)
    P, N, D = int(counts.sum()), n_out * (2 if swiglu else 1), 13
    assert P >= 3 * E and (n_out + 15) // 16 * E >= 4096 and K >= 1536
    g = synth.rng(318, E, n_out, K)
    q, s, gs = weights(g, (D, N, K), fmt)  # expert e has matrix e % D
    of = torch.arange(E, device="cuda") % D
    gsv = None if gs is None else (gs * (0.5 + np.arange(E) / E)).astype(np.float32)
    b = g.normal(0, 0.1, (E, N)).astype(np.float32) if bias else None
    bt = None if b is None else torch.from_numpy(b).cuda()
    if bias == "bf16":
        bt = bt.bfloat16()
        b = host(bt)
    x = synth.to_bf16_bits(g.standard_normal((P, K), dtype=np.float32))
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    sp = g.permutation(P).astype(np.int32)
    args = (bf16_dev(x), torch.from_numpy(q).cuda()[of], torch.from_numpy(s).cuda()[of], torch.from_numpy(offs).cuda(),
            torch.from_numpy(sp).cuda(), bt)
    kw = dict(fmt=FMTS[fmt], global_scales=None if gsv is None else torch.from_numpy(gsv).cuda(), swiglu=swiglu, out_dtype=out)
    y = mx.fp4_expert_matvec(*args, **kw)
    h, mag = np.empty((P, N)), np.empty((P, N))
    for d in range(D):
        w = V.weights_ref(q[d], s[d], None if gs is None else 1.0)
        for e in range(d, E, D):
            p = sp[offs[e]:offs[e + 1]]
            xe, c = V.bf16_to_f64(x[p]), 1.0 if gsv is None else float(gsv[e])
            h[p], mag[p] = xe @ w.T / c, np.abs(xe) @ np.abs(w).T / c
            if b is not None:
                h[p] += b[e]
    expert_of = np.empty(P, int)
    expert_of[sp] = np.repeat(np.arange(E), counts)
    ref, tol = with_swiglu(h, linear_bound(h, mag, K, None if b is None else b[expert_of]), swiglu)
    tol = tol + (2.0 ** -8 if out == torch.bfloat16 else U) * np.abs(ref) + 2.0 ** -133
    err = np.abs(host(y) - ref)
    assert y.shape == ref.shape and np.all(err <= tol), float((err / tol).max())
    assert torch.equal(y, mx.fp4_expert_matvec(*args, **kw))


def with_swiglu(h, tol, swiglu):
    """(reference, bound) behind the product's: silu has a slope of at most 1.1, its own evaluation errs by (|g| + 8) u."""
    if not swiglu:
        return h, tol
    ref = V.swiglu_ref(h)
    gate, up = np.split(h, 2, 1)
    tg, tu = np.split(tol, 2, 1)
    silu = gate / (1 + np.exp(-gate))
    return ref, 1.1 * tg * (np.abs(up) + tu) + np.abs(silu) * tu + (np.abs(gate) + 8) * U * np.abs(ref)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_the_decode_layers_products(fmt):
    """Both products of the decode layer (64 tokens, top-8 of 128, 1536 x 2048 with SwiGLU, then 2048 x 768) on the routing
    of random logits; the outputs of a sample of rows of W."""
    cfg = synth.MOE_CONFIGS["decode"]
    g = synth.rng(319)
    T, E, k = cfg.T, cfg.E, cfg.k
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids, _, offs, sp = mx.route(torch.randn(T, E, generator=gen, device="cuda"), k)
    idn = ids.cpu().numpy().reshape(-1)
    for N, K, swiglu, shared in ((2 * cfg.I, cfg.H, True, True), (cfg.H, cfg.I, False, False)):
        print(f"decode {fmt} {N} x {K}", flush=True)
        w = (torch.randn(E * N, K, generator=gen, device="cuda") * 0.02).bfloat16()
        gs = 448.0 / 0.02 if fmt == "nvfp4" else None
        q, s = (mx.nvfp4_quantize(w, gs, tiled=False) if gs else mx.quantize(w, tiled=False))[:2]
        q, s = q.view(E, N, -1), s.view(E, N, -1)
        x = synth.to_bf16_bits(g.standard_normal((T if shared else T * k, K), dtype=np.float32))
        gsd = None if gs is None else torch.full((E,), gs, device="cuda")
        y = host(mx.fp4_expert_matvec(bf16_dev(x), q, s, offs, sp, fmt=FMTS[fmt], global_scales=gsd, top_k=k if shared else 1,
                                      swiglu=swiglu, out_dtype=torch.float32))
        n_out = N // 2 if swiglu else N
        rows = np.unique(np.concatenate([[0, 15, 16, 31, 32, 63, 64, n_out - 1], g.integers(0, n_out, 12)]))
        at = torch.from_numpy(np.concatenate([rows, rows + n_out]) if swiglu else rows).cuda()
        qh, sh = q[:, at].cpu().numpy(), s[:, at].cpu().numpy()
        h, mag = V.expert_matvec_ref(x, qh, sh, idn.reshape(T, k), shared, None, None if gs is None else np.full(E, gs))
        ref, tol = with_swiglu(h, linear_bound(h, mag, K), swiglu)
        tol = tol + U * np.abs(ref) + 2.0 ** -133
        err = np.abs(y[:, rows] - ref)
        assert y.shape == (T * k, n_out) and np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("fmt", list(FMTS))
def test_more_pairs_than_a_tile_on_one_expert(fmt):
    expert(37, 9, 2, 40, 128, fmt, True, True, True, torch.float32, 1, crowd=True)
    expert(37, 9, 2, 40, 128, fmt, False, False, False, torch.float32, 1, crowd=True)


def test_last_expert_of_many_and_half_filled_groups():
    expert(2, 1024, 2, 16, 48, "nvfp4", False, True, True, torch.float32, 2)


def test_pairs_that_are_not_listed_keep_their_rows():
    args, kw, y = expert(6, 4, 2, 24, 64, "mxfp4", False, True, False, torch.float32, 3)
    offs, sp = args[3].clone(), args[4].clone()
    gone = sp[-1].item()
    offs[-1] -= 1  # the last pair is dropped
    if offs[-2] > offs[-1]:
        offs[-2] = offs[-1]
    out = torch.full_like(y, 7.0)
    z = mx.fp4_expert_matvec(*args[:3], offs, sp, **{k: v for k, v in kw.items() if k != "out_dtype"}, y=out)
    assert z is out
    keep = [p for p in range(12) if p != gone]
    assert torch.equal(z[keep], y[keep]) and bool((z[gone] == 7.0).all())


def test_bad_offsets_and_pairs_stay_inside():
    """Clamped or passed over: the kernel's own bounds, which the header states."""
    args, kw, y = expert(6, 4, 2, 24, 64, "mxfp4", False, True, False, torch.float32, 3)
    kw.pop("out_dtype")
    offs, sp = args[3], args[4].clone()
    sp[2], sp[5] = -1, 12
    dropped = sorted({args[4][2].item(), args[4][5].item()})
    keep = [p for p in range(12) if p not in dropped]
    z = mx.fp4_expert_matvec(*args[:3], offs, sp, **kw, y=torch.full_like(y, 7.0))
    assert torch.equal(z[keep], y[keep]) and bool((z[dropped] == 7.0).all())
    wide = offs.clone()
    wide[0], wide[-1] = -5, 1 << 30
    assert torch.equal(mx.fp4_expert_matvec(*args[:3], wide, args[4], **kw, y=torch.full_like(y, 7.0)), y)
    none = torch.zeros_like(offs)
    assert bool((mx.fp4_expert_matvec(*args[:3], none, sp, **kw, y=torch.full_like(y, 7.0)) == 7.0).all())


@pytest.mark.parametrize("fmt", list(FMTS))
def test_offsets_outside_the_pairs_with_fewer_pairs_than_experts(fmt):
    """An expert is one of those that have pairs by its clamped offsets, not by the offsets as given."""
    E, N, K, P = 70, 24, 64, 3
    g = synth.rng(317)
    q, s, _ = weights(g, (E, N, K), fmt)
    x = synth.to_bf16_bits(g.standard_normal((P, K), dtype=np.float32))
    args = bf16_dev(x), torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    kw = {"fmt": FMTS[fmt], "global_scales": torch.ones(E, device="cuda") if fmt == "nvfp4" else None}
    sp = torch.tensor([1, 2, 0], dtype=torch.int32, device="cuda")
    for good, bad in (([0] * 60 + [1] + [3] * 10, list(range(-60, 0)) + [1] + [3] * 10),
                      ([0] * 4 + [2, 3] + [3] * 65, [-9, -7, -7, 0, 2] + list(range(50, 116)))):
        y, z = (mx.fp4_expert_matvec(*args, torch.tensor(o, dtype=torch.int32, device="cuda"), sp, **kw,
                                     y=torch.full((P, N), 7.0, device="cuda")) for o in (good, bad))
        assert not (y == 7.0).all(1).any() and torch.equal(y, z)


def test_long_rows_and_many_rows():
    """K past the blocks that one round of waves takes; more rows of x than a grid has places for."""
    dense(2, 3, 1 << 18, "mxfp4", None, torch.float32, seed=6)
    dense(6, 5, (1 << 17) + 16, "nvfp4", "fp32", seed=6)
    g = synth.rng(314)
    M = (1 << 20) - 7
    q, s, _ = weights(g, (20, 32), "mxfp4")
    x = synth.to_bf16_bits(g.standard_normal((1000, 32), dtype=np.float32))
    xd = bf16_dev(x).repeat(M // 1000 + 1, 1)[:M]
    qd, sd = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    y = mx.fp4_matvec(xd, qd, sd)
    first = mx.fp4_matvec(xd[:1000], qd, sd)
    assert_dense(first, x, q, s, None, None, torch.bfloat16)
    ref, mag = V.matvec_ref(x, q, s)
    at = np.arange(M - 3000, M) % 1000
    err = np.abs(host(y[M - 3000:]) - ref[at])
    assert np.all(err <= linear_bound(ref[at], mag[at], 32) + 2.0 ** -8 * np.abs(ref[at]) + 2.0 ** -133)


def test_expert_weights_past_4_gib():
    """The last of 1024 experts' codes lie past 2^32 bytes, its scales past 2^28; two tokens choose it and the first."""
    E, N, K = 1024, 2056, 4096
    g = synth.rng(315)
    q0, s0, _ = weights(g, (2, N, K), "mxfp4")
    q = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(E, N, K // 32, dtype=torch.uint8, device="cuda")
    assert q.numel() > 1 << 32
    for i, e in enumerate((0, E - 1)):
        q[e], s[e] = torch.from_numpy(q0[i]).cuda(), torch.from_numpy(s0[i]).cuda()
    x = synth.to_bf16_bits(g.standard_normal((2, K), dtype=np.float32))
    ids = np.array([[E - 1, 0], [0, E - 1]])
    offs, sp = pairs_of(ids, E)
    y = mx.fp4_expert_matvec(bf16_dev(x), q, s, offs, sp, top_k=2, out_dtype=torch.float32)
    ref, mag = V.expert_matvec_ref(x, q0, s0, np.where(ids == 0, 0, 1), True)
    assert np.all(np.abs(host(y) - ref) <= linear_bound(ref, mag, K) + U * np.abs(ref))


def test_calls_on_two_streams_at_once_and_from_another_device(monkeypatch):
    xd, qd, sd, gs, y = dense(5, 300, 2048, "mxfp4", None, seed=7)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            got.append(mx.fp4_matvec(xd, qd, sd))
    torch.cuda.synchronize()
    assert all(torch.equal(t, y) for t in got)
    monkeypatch.setattr(mx.ops, "_current_gpu", lambda: -1)  # as if another device were the current one
    assert torch.equal(mx.fp4_matvec(xd, qd, sd), y)


def test_no_rows():
    q, s = torch.zeros(16, 32, dtype=torch.uint8, device="cuda"), torch.zeros(16, 2, dtype=torch.uint8, device="cuda")
    assert mx.fp4_matvec(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), q, s).shape == (0, 16)
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    y = mx.fp4_expert_matvec(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), q[None], s[None], i, i[:0], top_k=4)
    assert y.shape == (0, 16)


def test_another_stream_and_a_graph():
    xd, qd, sd, gs, y = dense(3, 200, 1024, "nvfp4", None, seed=5)
    args, kw, ye = expert(4, 16, 2, 64, 256, "mxfp4", True, True, True, seed=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = mx.fp4_matvec(xd, qd, sd, fmt=mx.FMT_NVFP4, global_scale=gs)
        b = mx.fp4_expert_matvec(*args, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, y) and torch.equal(b, ye)
    graphs = []
    for _ in range(2):  # two graphs share nothing but their inputs
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = (mx.fp4_matvec(xd, qd, sd, fmt=mx.FMT_NVFP4, global_scale=gs), mx.fp4_expert_matvec(*args, **kw))
        graphs.append((graph, out))
    x0, x1 = xd.clone(), -xd
    for i in range(4):
        xd.copy_(x1 if i % 2 else x0)
        eager = mx.fp4_matvec(xd, qd, sd, fmt=mx.FMT_NVFP4, global_scale=gs)
        for graph, out in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out[0], eager) and torch.equal(out[1], ye)


def test_refusals():
    z = lambda *s, d=torch.uint8: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    x, q, s = z(2, 64, d=bf), z(16, 32), z(16, 2)
    i2, p = z(2, d=torch.int32), z(2, d=torch.int32)
    bad = [lambda: mx.fp4_matvec(x.half(), q, s), lambda: mx.fp4_matvec(x[:, :32], q, s),
           lambda: mx.fp4_matvec(x, q, z(16, 4)), lambda: mx.fp4_matvec(x, q.cpu(), s),
           lambda: mx.fp4_matvec(x, q, s, fmt=mx.FMT_MXFP8), lambda: mx.fp4_matvec(x, q, s, global_scale=1.0),
           lambda: mx.fp4_matvec(x, q, z(16, 4), fmt=mx.FMT_NVFP4), lambda: mx.fp4_matvec(x, q, s, z(15, d=bf)),
           lambda: mx.fp4_matvec(x, q, s, z(16, d=torch.half)), lambda: mx.fp4_matvec(x, q, s, out_dtype=torch.half),
           lambda: mx.fp4_matvec(x[:1].expand(2, 64), q, s), lambda: mx.fp4_matvec(z(64, 2, d=bf).t(), q, s),
           lambda: mx.fp4_matvec(x, z(16, 64)[:, :32], s),
           lambda: mx.fp4_expert_matvec(x, q, s, i2, p), lambda: mx.fp4_expert_matvec(x, q[None], s[None], z(3, d=torch.int32), p),
           lambda: mx.fp4_expert_matvec(x, q[None], s[None], i2, p, top_k=2),
           lambda: mx.fp4_expert_matvec(x, q[None], s[None], i2.long(), p),
           lambda: mx.fp4_expert_matvec(x, z(1, 15, 32), z(1, 15, 2), i2, p, swiglu=True),
           lambda: mx.fp4_expert_matvec(x, q[None], s[None], i2, p, y=z(2, 15, d=bf)),
           lambda: mx.fp4_expert_matvec(x, q[None], z(1, 16, 4), i2, p, fmt=mx.FMT_NVFP4)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(mx.Mxfp4Error):  # rows 8-byte aligned
        mx.fp4_matvec(z(2, 68, d=bf)[:, 4:], q, s)
    with pytest.raises(mx.Mxfp4Error):
        mx.fp4_matvec(x, q, z(16, 4), fmt=mx.FMT_NVFP4, global_scale=-1.0)
