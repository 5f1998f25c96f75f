"""GPU parity of the block-quantized paged cache with the oracle: codes and scale bytes bit for bit, values read
back bit for bit (the MX formats' values are exact in bf16; NVFP4's are binary32 numbers, rounded once more)."""

import numpy as np
import pytest
import torch

import mixed_precision_moe_amd as mx
from mixed_precision_moe_amd import synth
from oracle import cache as C
from tests.gpu_common import bf16_dev, bf16_host_bits

pytestmark = pytest.mark.gpu
FMTS = {"mxfp4": mx.FMT_MXFP4, "nvfp4": mx.FMT_NVFP4, "mxfp8": mx.FMT_MXFP8}
GS = {"mxfp4": (1.0, 1.0), "nvfp4": (300.0, 77.5), "mxfp8": (1.0, 1.0)}


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Host:
    """The cache's memory as the oracle keeps it."""

    def __init__(self, cache, fmt):
        self.fmt = fmt
        d = self.d = cache.dims
        self.q = [cache.k_q.cpu().numpy().copy(), None if cache.v_q is None else cache.v_q.cpu().numpy().copy()]
        self.s = [cache.k_s.cpu().numpy().copy(), None if cache.v_s is None else cache.v_s.cpu().numpy().copy()]
        self.n = d.num_pages * d.page_size

    def flat(self, a):
        return a.reshape(self.n, *a.shape[2:])

    def write(self, planes, slots):
        for i, bits in enumerate(planes):
            if bits is None:
                continue
            q, s = C.encode_ref(bits, self.fmt, GS[self.fmt][i])
            for t, slot in enumerate(slots):
                if slot is not None and slot >= 0:
                    self.flat(self.q[i])[slot], self.flat(self.s[i])[slot] = q[t], s[t]

    def read(self, i, slots, fill):
        """bf16 bits; `fill` where the row belongs to no sequence."""
        v = C.bf16_bits(C.decode_ref(self.flat(self.q[i]), self.flat(self.s[i]), self.fmt, GS[self.fmt][i]))
        return np.stack([np.full(v.shape[1:], fill if slot is None else 0, np.uint16) if slot is None or slot < 0 else v[slot]
                         for slot in slots])

    def check(self, cache):
        for a, b in zip((cache.k_q, cache.v_q, cache.k_s, cache.v_s), self.q + self.s):
            if a is not None:
                np.testing.assert_array_equal(a.cpu().numpy(), b)


def make(fmt, pages, page, heads, k_dim, v_dim, seed=0):
    g = synth.rng(320, seed, pages, page)
    b = 16 if fmt == "nvfp4" else 32
    by = 1 if fmt == "mxfp8" else 2
    rnd = lambda d: torch.from_numpy(g.integers(0, 120, (pages, page, heads, d), dtype=np.uint8)).cuda() if d else None  # noqa: E731
    store = (rnd(k_dim // by), rnd(k_dim // b), rnd(v_dim // by), rnd(v_dim // b))
    c = mx.PagedCache(pages, page, heads, k_dim, v_dim, FMTS[fmt], *GS[fmt], storage=store)
    return c, Host(c, fmt), g


def rows_of(g, n, heads, dim, plain=True):
    if plain:
        return synth.to_bf16_bits(g.standard_normal((n, heads, dim)) * np.exp2(g.uniform(-6, 6, (n, heads, 1))))
    return synth.random_bits_matrix(n * heads, dim, int(g.integers(1 << 20))).reshape(n, heads, dim)


def cycle(fmt, page, heads, k_dim, v_dim, have, new, lead=0, tail=0, seed=0, holes=False, plain=True):
    """Writes `new` tokens a sequence after `have`, reads everything back, and compares memory and values."""
    print(f"cache {fmt} page={page} heads={heads} dims={k_dim},{v_dim} have={have} new={new} lead={lead} tail={tail}", flush=True)
    need = [-(-(h + n) // page) for h, n in zip(have, new)]
    pages = sum(need) + 2
    c, host, g = make(fmt, pages, page, heads, k_dim, v_dim, seed)
    order = list(g.permutation(pages))
    width = max(need + [1]) + 1
    table = np.full((len(have), width), -1, np.int32)
    for b, n in enumerate(need):
        table[b, :n] = [order.pop() for _ in range(n)]
    if holes:  # pages that are not there: no number, one past the last, far outside
        table[0, 0], table[-1, 0] = pages, -7
        if width > 2:
            table[0, 1] = np.iinfo(np.int32).max
    cu = lead + np.concatenate([[0], np.cumsum(new)])
    rows = int(cu[-1]) + tail
    kb = rows_of(g, rows, heads, k_dim, plain)
    vb = rows_of(g, rows, heads, v_dim, plain) if v_dim else None
    c.write(bf16_dev(kb), None if vb is None else bf16_dev(vb), i32(table), i32(cu), i32(have))
    slots = C.slots_ref(rows, cu, have, table, page, pages)
    host.write((kb, vb), slots)
    host.check(c)
    total = [h + n for h, n in zip(have, new)]
    cu = lead + np.concatenate([[0], np.cumsum(total)])
    rows = int(cu[-1]) + tail
    ko = torch.full((rows, heads, k_dim), 2.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full((rows, heads, v_dim), 2.0, dtype=torch.bfloat16, device="cuda") if v_dim else None
    k, v = c.read(i32(table), i32(cu), k_out=ko, v_out=vo)
    slots = C.slots_ref(rows, cu, None, table, page, pages)
    np.testing.assert_array_equal(bf16_host_bits(k), host.read(0, slots, 0x4000))
    if v_dim:
        np.testing.assert_array_equal(bf16_host_bits(v), host.read(1, slots, 0x4000))
    host.check(c)  # a read leaves the cache alone
    return c, host, table, cu


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("page,heads,k_dim,v_dim,have,new", [
    (16, 2, 64, 64, [0], [1]), (1, 1, 32, 32, [0, 3], [4, 1]), (16, 1, 32, 96, [5, 0, 31], [1, 1, 1]),
    (24, 8, 128, 128, [0, 0, 100], [70, 0, 3]), (64, 3, 96, 160, [63, 64, 65, 1], [1, 1, 1, 130]),
    (7, 5, 192, 0, [9, 2], [20, 6]), (128, 1, 576, 0, [1], [200]), (5, 16, 256, 224, [0, 11], [3, 9])])
def test_write_and_read_back(fmt, page, heads, k_dim, v_dim, have, new):
    cycle(fmt, page, heads, k_dim, v_dim, have, new)


def test_sixteen_element_heads():
    cycle("nvfp4", 16, 3, 16, 48, [4, 0], [5, 17])
    cycle("nvfp4", 16, 1, 16, 0, [4, 0], [5, 17])


@pytest.mark.parametrize("fmt", list(FMTS))
def test_rows_outside_every_sequence_are_left_alone(fmt):
    cycle(fmt, 8, 2, 64, 32, [3, 0, 9], [2, 0, 8], lead=3, tail=5)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_missing_pages(fmt):
    cycle(fmt, 4, 2, 64, 64, [6, 0, 2], [7, 9, 3], holes=True)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_arbitrary_patterns(fmt):
    """Every sign, exponent and mantissa, zero blocks among them."""
    cycle(fmt, 16, 2, 128, 64, [0, 0], [100, 61], plain=False)


def test_arbitrary_patterns_nvfp4():
    cycle("nvfp4", 16, 2, 128, 64, [0, 0], [100, 61], plain=False)


def test_many_sequences():
    g = np.random.default_rng(2)
    have, new = list(g.integers(0, 40, 300)), list(g.integers(0, 4, 300))
    cycle("mxfp8", 16, 1, 64, 32, have, new)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_many_rows(fmt):
    """Waves that take several rows: narrow ones, and more rows than waves are wanted, with sequences, gaps and missing
    pages inside a wave's rows."""
    g = np.random.default_rng(3)
    have, new = list(g.integers(0, 9, 900)), list(g.integers(0, 25, 900))
    cycle(fmt, 8, 1, 32, 32, have, new, lead=5, tail=9, holes=True)
    have, new = list(g.integers(0, 3, 41)), list(g.integers(1500, 2100, 41))
    cycle(fmt, 64, 1, 64, 32, have, new, holes=True, seed=1)


def test_the_widest_row():
    cycle("mxfp8", 2, 512, 2048, 0, [1], [2])
    cycle("nvfp4", 1, 1, 1 << 20, 16, [0], [2])


def test_codes_are_the_quantizers():
    """A cached row holds what quantize / nvfp4_quantize give for it."""
    g = synth.rng(321)
    bits = rows_of(g, 33, 4, 64)
    table, cu = i32([[2, 0, 1]]), i32([0, 33])
    for fmt in ("mxfp4", "nvfp4"):
        c = mx.PagedCache(3, 16, 4, 64, 0, FMTS[fmt], 9.0)
        c.write(bf16_dev(bits), None, table, cu)
        flat = bf16_dev(bits.reshape(33, 256))
        q, s, _ = mx.quantize(flat, tiled=False) if fmt == "mxfp4" else mx.nvfp4_quantize(flat, 9.0, tiled=False)
        at = [2 * 16 + i for i in range(16)] + list(range(16)) + [16]
        assert torch.equal(c.k_q.reshape(48, -1)[at], q) and torch.equal(c.k_s.reshape(48, -1)[at], s)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_strided_rows_and_heads(fmt):
    """Keys and values as slices of one fused projection, heads apart; written and read in place."""
    c, host, g = make(fmt, 4, 8, 3, 64, 32)
    kb, vb = rows_of(g, 19, 3, 64), rows_of(g, 19, 3, 32)
    fused = torch.full((19, 3, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, :, 8:72], fused[:, :, 104:] = bf16_dev(kb), bf16_dev(vb)
    table, cu = i32([[3, 1, 0]]), i32([0, 19])
    c.write(fused[:, :, 8:72], fused[:, :, 104:], table, cu)
    slots = C.slots_ref(19, [0, 19], None, [[3, 1, 0]], 8, 4)
    host.write((kb, vb), slots)
    host.check(c)
    out = torch.full((3, 19, 136), 2.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)  # heads outermost
    c.read(table, cu, k_out=out[:, :, :64], v_out=out[:, :, 72:104])
    np.testing.assert_array_equal(bf16_host_bits(out[:, :, :64].contiguous()), host.read(0, slots, 0))
    np.testing.assert_array_equal(bf16_host_bits(out[:, :, 72:104].contiguous()), host.read(1, slots, 0))
    assert bool((out[:, :, 64:72] == 2.0).all()) and bool((out[:, :, 104:] == 2.0).all())


def test_windows_and_wide_tables():
    """Reading the last positions of each sequence; a table that is a slice of a wider one."""
    c, host, table, cu = cycle("mxfp4", 4, 2, 64, 64, [0, 0], [30, 9])
    wide = i32(np.pad(table, ((0, 0), (0, 5)), constant_values=1 << 20))[:, :table.shape[1]]
    start = [22, 3]
    k, v = c.read(wide, i32([0, 8, 14]), i32(start), rows=14)
    slots = C.slots_ref(14, [0, 8, 14], start, table, 4, c.dims.num_pages)
    np.testing.assert_array_equal(bf16_host_bits(k), host.read(0, slots, 0))
    # positions before the first and past the table read as zeros
    k, v = c.read(wide, i32([0, 3, 5]), i32([-2, 4 * table.shape[1] - 1]), rows=5)
    got = bf16_host_bits(k)
    assert not got[:2].any() and not got[4].any()
    np.testing.assert_array_equal(got, host.read(0, C.slots_ref(5, [0, 3, 5], [-2, 4 * table.shape[1] - 1], table, 4, c.dims.num_pages), 0))


def all_nvfp4_values(gs):
    """A one-plane NVFP4 cache of every code under every finite scale, and its values in float64."""
    s = np.arange(254, dtype=np.uint8)
    s[127:] += 1  # 0x7F and 0xFF are NaN
    q = np.tile(np.arange(16, dtype=np.uint8).reshape(8, 2) @ np.array([1, 16], np.uint8), (254, 1))
    store = [torch.from_numpy(t.reshape(2, 127, 1, -1)).cuda() for t in (q, s)]
    c = mx.PagedCache(2, 127, 1, 16, 0, mx.FMT_NVFP4, gs, storage=(*store, None, None))
    code = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
    m, e = np.minimum(s & 127, 126), (s & 127) >> 3
    scale = np.where(e > 0, np.ldexp(8.0 + m % 8, e.astype(int) - 10), np.ldexp(m % 8.0, -9)) * np.where(s & 128, -1, 1)
    with np.errstate(over="ignore"):
        v = code[None, :] * scale[:, None] / float(np.float32(gs))
    k, _ = c.read(i32([[0, 1]]), i32([0, 254]), rows=254)
    return k.view(254, 16).double().cpu().numpy(), v


@pytest.mark.parametrize("k", [-149, -140, -126, -120, -1, 0, 60, 100, 118, 120, 127])
def test_nvfp4_values_under_a_power_of_two(k):
    """A power of two as global scale moves the exponent and nothing else (values have six bits), also one under which a
    scale alone would overflow; past bf16's range there are infinities, below it the steps of 2^-133."""
    got, v = all_nvfp4_values(2.0 ** k)
    with np.errstate(over="ignore"):
        want = np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), np.where(np.abs(v) < 2.0 ** -126, np.rint(v * 2.0 ** 133) * 2.0 ** -133, v))
    np.testing.assert_array_equal(got, want)
    assert k in (-149, -140) or np.isfinite(got).any() and got.any()


@pytest.mark.parametrize("gs", [1.4e-45, 3e-39, 1.1e-36, 2.3e-36, 0.0137, 512 / 257, 512 / 285, 0.99999994, 1.0000001, 77.123, 448.0 / 0.02, 2.9e30, 3.4e38])
def test_nvfp4_values_under_any_global_scale(gs):
    """The quotient and its product with the code are rounded to binary32 (2^-24 each; below its normal range 2^-150 and six
    times that), then once to bf16: 2^-8 of the value bounds half a step, 2^-134 it below the normal range."""
    got, v = all_nvfp4_values(gs)
    top = (2 - 2.0 ** -7) * 2.0 ** 127
    with np.errstate(invalid="ignore"):
        near = np.abs(got - v) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(v) + 2.0 ** -134 + 2.0 ** -147
    assert np.all(np.where(np.abs(v) > top, np.abs(got) >= top, near))
    assert not got[np.isnan(got)].size and np.all(np.signbit(got) == np.signbit(v))


def test_offsets_past_32_bits():
    """Slots whose bytes lie past 4 GiB of a plane, and a slot number times its elements past 2^32."""
    pages, page, heads, dim = 18000, 64, 32, 128  # 4.7e9 elements, 2.4e9 bytes of codes; MXFP8: 4.7e9 bytes
    c = mx.PagedCache(pages, page, heads, dim, 0, mx.FMT_MXFP8)
    g = synth.rng(322)
    bits = rows_of(g, 70, heads, dim)
    table, cu = i32([[pages - 1, 0]]), i32([0, 70])
    c.write(bf16_dev(bits), None, table, cu)
    q, s = C.encode_ref(bits, "mxfp8", 1.0)
    np.testing.assert_array_equal(c.k_q[pages - 1].cpu().numpy(), q[:64])
    np.testing.assert_array_equal(c.k_s[pages - 1].cpu().numpy(), s[:64])
    np.testing.assert_array_equal(c.k_q[0, :6].cpu().numpy(), q[64:])
    k, _ = c.read(table, cu, rows=70)
    np.testing.assert_array_equal(bf16_host_bits(k), C.bf16_bits(C.decode_ref(q, s, "mxfp8", 1.0)))
    assert not c.k_q[1:pages - 1].any()


def test_nothing_to_do():
    c = mx.PagedCache(2, 4, 1, 32, 32, mx.FMT_MXFP4)
    z = torch.zeros(0, 1, 32, dtype=torch.bfloat16, device="cuda")
    c.write(z, z, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), i32([0]))
    c.write(z, z, i32([[0]]), i32([0, 0]))
    k, v = c.read(i32([[0]]), i32([0, 0]), rows=0)
    assert k.shape == (0, 1, 32)
    x = torch.ones(3, 1, 32, dtype=torch.bfloat16, device="cuda")
    c.write(x, x, torch.zeros(1, 0, dtype=torch.int32, device="cuda"), i32([0, 3]))  # a table without pages
    empty = mx.PagedCache(0, 4, 1, 32, 32, mx.FMT_MXFP4)
    empty.write(x, x, i32([[0]]), i32([0, 3]))
    assert not c.k_q.any() and not empty.read(i32([[0]]), i32([0, 3]), rows=3)[0].any()


def test_another_stream_and_a_graph():
    c, host, g = make("nvfp4", 6, 8, 2, 64, 64)
    kb, vb = rows_of(g, 11, 2, 64), rows_of(g, 11, 2, 64)
    k, v, table, cu, start = bf16_dev(kb), bf16_dev(vb), i32([[5, 0], [2, 4]]), i32([0, 9, 11]), i32([1, 6])
    cu_all = i32([0, 10, 18])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.write(k, v, table, cu, start)
        got = c.read(table, cu_all, rows=18)
    torch.cuda.current_stream().wait_stream(s)
    host.write((kb, vb), C.slots_ref(11, [0, 9, 11], [1, 6], [[5, 0], [2, 4]], 8, 6))
    host.check(c)
    slots = C.slots_ref(18, [0, 10, 18], None, [[5, 0], [2, 4]], 8, 6)
    np.testing.assert_array_equal(bf16_host_bits(got[0]), host.read(0, slots, 0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.write(k, v, table, cu, start)
        out = c.read(table, cu_all, rows=18)
    for i in range(4):  # new rows and positions on every replay
        kb = rows_of(g, 11, 2, 64)
        k.copy_(bf16_dev(kb))
        start.copy_(i32([i, 6 - i]))
        graph.replay()
        torch.cuda.synchronize()
        host.write((kb, vb), C.slots_ref(11, [0, 9, 11], [i, 6 - i], [[5, 0], [2, 4]], 8, 6))
        host.check(c)
        np.testing.assert_array_equal(bf16_host_bits(out[0]), host.read(0, slots, 0))
        eager = c.read(table, cu_all, rows=18)
        assert torch.equal(eager[0], out[0]) and torch.equal(eager[1], out[1])


def test_calls_from_another_device(monkeypatch):
    c, host, g = make("mxfp4", 3, 4, 2, 32, 32)
    kb, vb = rows_of(g, 5, 2, 32), rows_of(g, 5, 2, 32)
    monkeypatch.setattr(mx.ops, "_current_gpu", lambda: -1)  # as if another device were the current one
    c.write(bf16_dev(kb), bf16_dev(vb), i32([[2, 1]]), i32([0, 5]))
    slots = C.slots_ref(5, [0, 5], None, [[2, 1]], 4, 3)
    host.write((kb, vb), slots)
    host.check(c)
    np.testing.assert_array_equal(bf16_host_bits(c.read(i32([[2, 1]]), i32([0, 5]), rows=5)[1]), host.read(1, slots, 0))


def test_refusals():
    c = mx.PagedCache(4, 8, 2, 64, 32, mx.FMT_MXFP4)
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    k, v, t, cu = z(3, 2, 64), z(3, 2, 32), i32([[0]]), i32([0, 3])
    bad = [lambda: c.write(k.float(), v, t, cu), lambda: c.write(k, None, t, cu), lambda: c.write(k[:, :1], v, t, cu),
           lambda: c.write(k, v[:2], t, cu), lambda: c.write(k, v, t.long(), cu), lambda: c.write(k, v, t, cu[:1]),
           lambda: c.write(k, v, t, cu, i32([0, 0])), lambda: c.write(k, v, t.cpu(), cu), lambda: c.write(k.cpu(), v, t, cu),
           lambda: c.write(k, v, i32([[0, 1]]).t().expand(2, 2).t()[:2], i32([0, 1, 3])),
           lambda: c.write(z(3, 64, 2).transpose(1, 2), v, t, cu), lambda: c.read(t, cu), lambda: c.read(t, cu, rows=-1),
           lambda: c.read(t, cu, rows=2, k_out=k, v_out=v), lambda: c.read(t, cu, k_out=k),
           lambda: c.read(t, cu, rows=3, v_out=v)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(mx.Mxfp4Error):  # rows 8-byte aligned
        c.write(z(3, 2, 68)[:, :, 4:], v, t, cu)
