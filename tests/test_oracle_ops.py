"""Pins of the oracle's balance loss, 4-bit products and paged cache against hand values, brute force and
difference quotients."""

import math
from fractions import Fraction

import numpy as np
import pytest

from mixed_precision_moe_amd import synth
from oracle import balance as B
from oracle import cache as C
from oracle import linear as L
from oracle import matvec as V
from oracle import quant as Q


def test_balance_hand_values():
    # two experts, uniform probabilities, three pairs to expert 0 and one to expert 1: 2 / (1 * 16) * (3 * 2 + 1 * 2) = 1
    loss, counts, grad = B.balance_ref(np.zeros((4, 2)), [[0], [0], [0], [1]])
    assert loss == 1.0 and list(counts) == [3, 1]
    # d = 1/8 * (1, -1), p = 1/2: +-1/16
    np.testing.assert_array_equal(grad, np.tile([1 / 16, -1 / 16], (4, 1)))
    # all of it on one expert, which everything chose: E
    l = np.full((5, 8), -np.inf)
    l[:, 3] = 0.0
    loss, counts, grad = B.balance_ref(l, np.full((5, 1), 3))
    assert loss == 8.0 and counts[3] == 5 and not grad.any()
    loss, counts, grad = B.balance_ref(np.zeros((3, 4)), np.zeros((3, 2), int), np.zeros(3, bool))
    assert loss == 0.0 and not counts.any() and not grad.any()


def test_balance_brute_force_and_masks():
    g = synth.rng(200)
    l = g.standard_normal((9, 6)) * 2
    ids = np.array([g.permutation(6)[:2] for _ in range(9)])
    ids[4, 1] = -1  # a dropped pair
    ids[5, 0] = 6
    mask = g.random(9) < 0.6
    l[~mask] = np.nan
    loss, counts, grad = B.balance_ref(l, ids, mask, g=0.25)
    V_, total, n = 0, 0.0, [0] * 6
    for t in range(9):
        if mask[t]:
            V_ += 1
            for e in ids[t]:
                if 0 <= e < 6:
                    n[e] += 1
    for e in range(6):
        total += n[e] * math.fsum(math.exp(l[t, e]) / math.fsum(math.exp(v) for v in l[t]) for t in range(9) if mask[t])
    assert list(counts) == n
    assert loss == pytest.approx(6 / (2 * V_ * V_) * total, rel=1e-13)
    assert not grad[~mask].any()
    # difference quotients: f is smooth, h^2 |f'''| is below 1e-9 of f at h = 1e-4
    for t, e in zip(np.flatnonzero(mask), [0, 3, 5, 1, 2, 4, 0, 1, 2]):
        a, b = l.copy(), l.copy()
        a[t, e] += 1e-4
        b[t, e] -= 1e-4
        d = (B.balance_ref(a, ids, mask)[0] - B.balance_ref(b, ids, mask)[0]) / 2e-4
        assert 0.25 * d == pytest.approx(grad[t, e], abs=1e-9)


def test_matvec_equals_the_linear_oracle_and_brute_force():
    g = synth.rng(201)
    x = synth.to_bf16_bits(g.standard_normal((3, 64)))
    w = synth.to_bf16_bits(g.standard_normal((5, 64)) * 0.02)
    q, s = Q.quantize_ref(w)
    np.testing.assert_allclose(V.matvec_ref(x, q, s)[0], L.linear_bruteforce(x, q, s), rtol=1e-13)
    gs = 1234.5
    q, s = Q.nvfp4_quantize_ref(w, gs)
    y, mag = V.matvec_ref(x, q, s, np.arange(5.0), gs)
    for m in range(3):
        for n in range(5):
            terms = []
            for k in range(64):
                c = int(q[n, k // 2]) >> (4 * (k % 2)) & 15
                v = (0, .5, 1, 1.5, 2, 3, 4, 6)[c & 7] * (-1 if c & 8 else 1) * float(Q.E4M3_MAGNITUDES[s[n, k // 16]])
                terms.append(v / gs * float(Q.bf16_to_f64(x[m, k])))
            assert y[m, n] == pytest.approx(math.fsum(terms) + n, rel=1e-12, abs=1e-12)
            assert mag[m, n] == pytest.approx(math.fsum(map(abs, terms)), rel=1e-12)


def test_expert_products_are_the_dense_ones_row_by_row():
    g = synth.rng(202)
    E, N, K = 3, 6, 32
    q = np.stack([Q.quantize_ref(synth.to_bf16_bits(g.standard_normal((N, K))))[0] for _ in range(E)])
    s = np.full((E, N, 1), 127, np.uint8)
    x = synth.to_bf16_bits(g.standard_normal((2, K)))
    ids = np.array([[2, 0], [1, 2]])
    y, _ = V.expert_matvec_ref(x, q, s, ids, True)
    for p, (t, e) in enumerate(((0, 2), (0, 0), (1, 1), (1, 2))):
        np.testing.assert_array_equal(y[p], V.matvec_ref(x[t:t + 1], q[e], s[e])[0][0])
    h = np.array([[0.0, 1.0, 3.0, 4.0]])
    np.testing.assert_allclose(V.swiglu_ref(h), [[0.0, 4.0 / (1 + math.exp(-1.0))]])


def test_cache_slots_by_hand():
    # sequence 0: positions 3, 4 (pages 7, 2 of four tokens); sequence 1: none; sequence 2: positions 0, 1, page missing
    got = C.slots_ref(6, [1, 3, 3, 5], [3, 0, 0], [[7, 2], [0, 0], [-1, 5]], 4, 8)
    assert got == [None, 7 * 4 + 3, 2 * 4 + 0, -1, -1, None]
    assert C.slots_ref(3, [0, 3], None, [[9, 1]], 2, 9) == [-1, -1, 2]
    assert C.slots_ref(2, [0, 2], [-1], [[0]], 1, 1) == [-1, 0]


@pytest.mark.parametrize("fmt,gs", [("mxfp4", 1.0), ("nvfp4", 40.0), ("mxfp8", 1.0)])
def test_cache_values_are_near_what_was_written(fmt, gs):
    g = synth.rng(203)
    bits = synth.to_bf16_bits(g.standard_normal((4, 2, 96)))
    v = Q.bf16_to_f64(bits)
    q, s = C.encode_ref(bits, fmt, gs)
    assert q.shape == (4, 2, 96 if fmt == "mxfp8" else 48) and s.shape == (4, 2, 96 // (16 if fmt == "nvfp4" else 32))
    got = C.decode_ref(q, s, fmt, gs)
    b = 16 if fmt == "nvfp4" else 32
    top = np.repeat(np.abs(v).reshape(4, 2, -1, b).max(-1), b, -1)
    # half the widest step: a sixth of the block's maximum in E2M1 (saturation and the scale's own rounding add
    # an eighth and 2^-4), 2^-4 of the value in E4M3
    assert np.all(np.abs(got - v) <= (2.0 ** -4 * np.abs(v) + 2.0 ** -10 * top if fmt == "mxfp8" else top * (1 / 6 + 1 / 8 + 2.0 ** -4)))


def nearest_bf16(v):
    """The bf16 number nearest to the fraction v >= 0 in bf16's normal range, the even one of two."""
    e = 0
    while v >= Fraction(2) ** (e + 1):
        e += 1
    while v < Fraction(2) ** e:
        e -= 1
    return round(v / Fraction(2) ** (e - 7)) * Fraction(2) ** (e - 7)


# scale / global scale a hair off a midpoint of bf16: binary32 on the way rounds it onto the midpoint, or past it
@pytest.mark.parametrize("gs", [8 * 64 / 257, 8 * 64 / 261, 8 * 64 / 285, 27 * 64 / 509, 45 * 64 / 371, 300.0, 0.3, 1e-30, 1e30])
def test_cache_values_are_the_definition_rounded_once(gs):
    gs = float(np.float32(gs))
    q = np.tile(np.arange(16, dtype=np.uint8).reshape(8, 2) @ np.array([1, 16], np.uint8), (127, 1))
    got = C.bf16_bits(C.decode_ref(q, np.arange(127, dtype=np.uint8)[:, None], "nvfp4", gs))
    mags = [Fraction(0), Fraction(1, 2), Fraction(1), Fraction(3, 2), Fraction(2), Fraction(3), Fraction(4), Fraction(6)]
    for s in range(127):
        m, e = s % 8, s // 8
        scale = Fraction(8 + m if e else m, 8) * Fraction(2) ** (max(e, 1) - 7)
        for code in range(16):
            v = mags[code % 8] * scale / Fraction(gs)
            want = float(nearest_bf16(v)) if v else 0.0
            bits = int(np.float32(want).view(np.uint32)) >> 16 | (0x8000 if code >= 8 else 0)
            assert got[s, code] == bits, (s, code)


def test_bf16_rounding_is_to_nearest_even():
    v = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -2.0, 3.4e38, np.inf, -0.0], np.float32)
    assert list(C.bf16_bits(v)) == [0x3F80, 0x3F80, 0x3F82, 0xC000, 0x7F80, 0x7F80, 0x8000]
