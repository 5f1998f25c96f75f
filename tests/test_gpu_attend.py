"""GPU parity of the attention over the paged cache with the float64 oracle.

Tolerance, per element of the result: the weights p are rounded to bf16 (half a step, 2^-8 of each), their exponents carry
the products' error (dim products and sums in binary32, each 2^-24 of the sum of magnitudes at most, and half as many again
for the matrix instruction's own order) and that of scaling, subtracting the maximum and the hardware's exponential
(2^-24 of the exponent each, 2^-22 of the result), the sums run over as many terms as the row sees (2^-24 of the
magnitudes each); the whole is rounded to the type once."""

import numpy as np
import pytest
import torch

import mixed_precision_moe_amd as mx
from mixed_precision_moe_amd import synth
from oracle import attend as A
from oracle import cache as C
from tests.gpu_common import bf16_dev, bf16_host_f64

pytestmark = pytest.mark.gpu
FMTS = {"mxfp4": mx.FMT_MXFP4, "nvfp4": mx.FMT_NVFP4, "mxfp8": mx.FMT_MXFP8}
GS = {"mxfp4": (1.0, 1.0), "nvfp4": (300.0, 77.5), "mxfp8": (1.0, 1.0)}


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def tolerance(out, weight, score, dim, seen, half_step):
    exponent = score * (1.5 * dim + 4) * 2.0 ** -24 + 2.0 ** -22
    return weight * (2.0 ** -8 + 2 * exponent[..., None] + seen * 2.0 ** -23) + np.abs(out) * half_step + 1e-30


class Setup:
    """A cache filled through `write`, with ragged sequences and pages in random order."""

    def __init__(self, fmt, page, heads, k_dim, v_dim, have, new, group=1, lead=0, tail=0, seed=0, spare=2):
        print(f"attend {fmt} page={page} heads={heads}x{group} dims={k_dim},{v_dim} have={have} new={new} lead={lead} tail={tail}",
              flush=True)
        g = self.g = synth.rng(340, seed, page, k_dim)
        self.fmt, self.page, self.have, self.new = fmt, page, have, new
        need = [-(-(h + n) // page) for h, n in zip(have, new)]
        pages = sum(need) + spare
        by, block = (1 if fmt == "mxfp8" else 2), (16 if fmt == "nvfp4" else 32)
        # what no sequence holds is arbitrary, NaN among it
        rnd = lambda d: torch.from_numpy(g.integers(0, 256, (pages, page, heads, d), dtype=np.uint8)).cuda()  # noqa: E731
        store = (rnd(k_dim // by), rnd(k_dim // block), rnd(v_dim // by), rnd(v_dim // block))
        self.cache = mx.PagedCache(pages, page, heads, k_dim, v_dim, FMTS[fmt], *GS[fmt], storage=store)
        order = list(g.permutation(pages))
        self.table = np.full((len(have), max(need + [1])), -1, np.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = [order.pop() for _ in range(n)]
        total = [h + n for h, n in zip(have, new)]
        kv = [bf16_dev(synth.to_bf16_bits(g.standard_normal((sum(total), heads, d)) * np.exp2(g.uniform(-1, 1, (sum(total), heads, 1)))))
              for d in (k_dim, v_dim)]
        self.cache.write(*kv, i32(self.table), i32(np.concatenate([[0], np.cumsum(total)])))
        self.cu = lead + np.concatenate([[0], np.cumsum(new)])
        self.rows = int(self.cu[-1]) + tail
        self.q = bf16_dev(synth.to_bf16_bits(g.standard_normal((self.rows, heads * group, k_dim))))

    def values(self):
        c, n = self.cache, self.cache.dims.num_pages * self.page
        out = []
        for q, s, gs in ((c.k_q, c.k_s, GS[self.fmt][0]), (c.v_q, c.v_s, GS[self.fmt][1])):
            q, s = (t.cpu().numpy().reshape(n, t.shape[2], -1) for t in (q, s))
            # the oracle knows the codes and scales that the quantizers write; others are no numbers here
            with np.errstate(all="ignore"):
                if self.fmt == "nvfp4":
                    v = np.where(np.repeat(s, 16, axis=-1) > 126, np.nan, C.decode_ref(q, np.minimum(s, 126), self.fmt, gs))
                elif self.fmt == "mxfp8":
                    none = ((q & 127) == 127) | (np.repeat(s, 32, axis=-1) == 255)
                    v = np.where(none, np.nan, C.decode_ref(np.where(none, 0, q).astype(np.uint8), s, self.fmt, gs))
                else:
                    v = np.where(np.repeat(s, 32, axis=-1) == 255, np.nan, C.decode_ref(q, s, self.fmt, gs))
            out.append(v)
        return out

    def args(self):
        return i32(self.table), i32(self.cu), i32(self.have)

    def check(self, got, mask=None, scale=None, table=None, start=None, fill=None, half_step=2.0 ** -8, rows=None):
        with np.errstate(all="ignore"):
            out, weight, score = A.attend_ref(bf16_host_f64(self.q), *self.values(), self.cu, self.have if start is None else start,
                                              self.table if table is None else table, self.page, mask, scale)
        got = got.double().cpu().numpy()
        none = np.isnan(out[:, 0, 0])
        if fill is not None:
            assert np.all(got[none] == fill)
        dim = self.q.shape[2]
        tol = tolerance(out, weight, score, dim, max(self.have + [0]) + max(self.new + [0]), half_step)
        off = np.abs(got - out)
        assert np.all(off[~none] <= tol[~none]), float(np.nanmax((off / tol)[~none]))


def tree_mask(g, new, rows, lead, W=None):
    """Each draft sees itself and its ancestors of a random tree."""
    W = max(new) if W is None else W
    mask, at = np.zeros((rows, W), bool), lead
    for n in new:
        for i in range(n):
            if i:
                mask[at + i] = mask[at + g.integers(0, i)]
            if i < W:
                mask[at + i, i] = True
        at += n
    return mask


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("page,heads,group,k_dim,v_dim,have,new", [
    (16, 2, 1, 64, 64, [0], [1]), (16, 2, 4, 64, 64, [77], [1]), (1, 1, 3, 32, 32, [0, 3], [4, 1]),
    (24, 1, 16, 128, 128, [31, 0, 200], [1, 1, 1]), (64, 3, 5, 96, 160, [63, 64, 65, 127, 128, 129], [1, 2, 1, 1, 3, 1]),
    (32, 2, 8, 192, 128, [300, 5], [1, 9]), (7, 5, 2, 256, 224, [130, 0, 1], [3, 20, 0]), (128, 1, 1, 256, 256, [500], [2]),
    (5, 8, 1, 32, 256, [0, 11], [3, 9]), (16, 1, 7, 128, 64, [0, 0, 0], [50, 1, 0])])
def test_rows_up_to_their_own_position(fmt, page, heads, group, k_dim, v_dim, have, new):
    s = Setup(fmt, page, heads, k_dim, v_dim, have, new, group)
    s.check(s.cache.attend(s.q, *s.args()))


@pytest.mark.parametrize("k_dim,v_dim", [(16, 16), (48, 80), (112, 144), (176, 208), (240, 16)])
def test_dimensions_of_sixteen(k_dim, v_dim):
    s = Setup("nvfp4", 16, 3, k_dim, v_dim, [40, 0, 150], [3, 17, 1], 2)
    s.check(s.cache.attend(s.q, *s.args()))


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("new,group", [([1, 1], 16), ([5, 2, 9], 1), ([33, 0, 12], 3), ([64, 17], 2), ([3, 40, 1], 8), ([150], 4)])
def test_trees_of_drafts(fmt, new, group):
    g = np.random.default_rng(sum(new))
    have = [int(x) for x in g.integers(0, 300, len(new))]
    s = Setup(fmt, 24, 2, 128, 64, have, new, group, lead=2, tail=3)
    mask = tree_mask(s.g, new, s.rows, 2)
    out = torch.full((s.rows, 2 * group, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    s.check(s.cache.attend(s.q, *s.args(), tree_mask=torch.from_numpy(mask).cuda(), out=out), mask, fill=7.0)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_long_contexts_and_many_parts(fmt):
    """Contexts that many workers share, beside short ones."""
    s = Setup(fmt, 64, 1, 64, 64, [9000, 3, 0, 2500], [2, 1, 1, 5], 2)
    s.check(s.cache.attend(s.q, *s.args()))


def test_many_sequences():
    g = np.random.default_rng(5)
    have, new = [int(x) for x in g.integers(0, 90, 300)], [int(x) for x in g.integers(0, 4, 300)]
    s = Setup("mxfp8", 16, 1, 32, 32, have, new, 2)
    s.check(s.cache.attend(s.q, *s.args()))
    mask = tree_mask(s.g, new, s.rows, 0)
    s.check(s.cache.attend(s.q, *s.args(), tree_mask=torch.from_numpy(mask).cuda()), mask)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_rows_that_see_nothing_and_empty_masks(fmt):
    s = Setup(fmt, 8, 2, 64, 64, [0, 0, 20], [6, 1, 4], 2)
    mask = tree_mask(s.g, s.new, s.rows, 0)
    mask[[0, 3, 6]] = False  # two rows of the first sequence and the only one of the second
    mask[7] = False          # one that still sees its context
    got = s.cache.attend(s.q, *s.args(), tree_mask=torch.from_numpy(mask).cuda())
    s.check(got, mask)
    assert not got[[0, 3, 6]].any() and got[7].any()
    for none in (np.zeros((s.rows, 0), bool), np.zeros((s.rows, 3), bool)):
        s.check(s.cache.attend(s.q, *s.args(), tree_mask=torch.from_numpy(none).cuda()), none)


def test_masks_narrower_and_wider_than_the_drafts():
    s = Setup("mxfp8", 16, 2, 64, 64, [10, 50], [9, 3], 2)
    for W in (4, 30):
        mask = tree_mask(s.g, s.new, s.rows, 0, W)
        mask[:, 9:] = True  # no such drafts
        wide = torch.zeros(s.rows, 64, dtype=torch.uint8, device="cuda")
        wide[:, 5:5 + W] = torch.from_numpy(mask).cuda() * 200
        s.check(s.cache.attend(s.q, *s.args(), tree_mask=wide[:, 5:5 + W]), mask)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_positions_without_pages(fmt):
    s = Setup(fmt, 4, 2, 64, 64, [30, 2, 200], [3, 9, 2], 3)
    n = s.cache.dims.num_pages
    table = s.table.copy()
    table[0, 0], table[0, 3], table[1, 0], table[2, 20:25] = n, -7, -1, np.iinfo(np.int32).max
    s.check(s.cache.attend(s.q, i32(table), *s.args()[1:]), table=table)
    # a table that ends before the positions do, and one without columns
    s.check(s.cache.attend(s.q, i32(table[:, :2]), *s.args()[1:]), table=table[:, :2])
    assert not s.cache.attend(s.q, i32(table[:, :0]), *s.args()[1:]).any()
    # positions before the first
    start = [-2, -9, -40]
    s.check(s.cache.attend(s.q, i32(s.table), i32(s.cu), i32(start)), start=start)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_nan_in_hidden_places(fmt):
    """A draft whose keys and values are not numbers reaches those rows alone that see it."""
    s = Setup(fmt, 16, 2, 128, 128, [20, 3], [8, 5], 2)
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    mask = tree_mask(s.g, s.new, s.rows, 0)
    mask[:, 2] = False
    mask[2, 2] = True  # seen by itself alone
    for pos, plane in ((22, "k"), (22, "v")):
        page, slot = s.table[0, pos // 16], pos % 16
        getattr(s.cache, plane + "_s")[page, slot, 0] = nan
        if fmt == "mxfp8":
            getattr(s.cache, plane + "_q")[page, slot, 1] = 0x7F
    got = s.cache.attend(s.q, *s.args(), tree_mask=torch.from_numpy(mask).cuda())
    rows = [t for t in range(s.rows) if t != 2]
    clean = mask.copy()
    clean[2] = False
    with np.errstate(all="ignore"):
        out, weight, score = A.attend_ref(bf16_host_f64(s.q), *s.values(), s.cu, s.have, s.table, 16, clean)
    tol = tolerance(out, weight, score, 128, 28, 2.0 ** -8)
    assert np.all(np.abs(got.double().cpu().numpy() - out)[rows] <= tol[rows])
    assert bool(torch.isnan(got[2, :2]).all())  # the query heads of key head 0
    # values alone
    getattr(s.cache, "k_s")[s.table[0, 1], 6, 0] = 100
    got = s.cache.attend(s.q, *s.args(), tree_mask=torch.from_numpy(mask).cuda())
    assert np.all(np.abs(got.double().cpu().numpy() - out)[rows] <= tol[rows]) and bool(torch.isnan(got[2, :2]).any())


def test_scales():
    for scale in (0.0, -0.3, 1.0, 7.5):
        s = Setup("mxfp4", 16, 2, 64, 64, [70, 3], [3, 2], 2)
        s.check(s.cache.attend(s.q, *s.args(), scale=scale), scale=scale)


def test_large_scores_keep_their_order():
    """Scores far apart: all weight on one position, also where the maximum comes last or first."""
    s = Setup("mxfp8", 32, 1, 64, 64, [400], [1], 1)
    for pos in (0, 127, 128, 399, 400):
        q = s.values()[0][s.table[0, pos // 32] * 32 + pos % 32, 0]
        s.q = bf16_dev(synth.to_bf16_bits(np.sign(q)[None, None] * 8))
        s.check(s.cache.attend(s.q, *s.args(), scale=4.0), scale=4.0)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_float_results_strides_and_outputs(fmt):
    s = Setup(fmt, 16, 2, 64, 96, [33, 5, 200], [2, 1, 3], 3, lead=1, tail=1)
    s.check(s.cache.attend(s.q, *s.args(), out_dtype=torch.float32), half_step=2.0 ** -24)
    # queries as slices of a fused projection, heads outermost in the result
    fused = torch.full((s.rows, 6, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, :, 8:72] = s.q
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((6, s.rows, 128), 3.0, dtype=dtype, device="cuda").transpose(0, 1)
        got = s.cache.attend(fused[:, :, 8:72], *s.args(), out=out[:, :, 8:104])
        s.check(got, fill=3.0)
        assert bool((out[:, :, :8] == 3.0).all()) and bool((out[:, :, 104:] == 3.0).all())


def test_no_start_and_a_slice_of_a_wider_table():
    s = Setup("nvfp4", 8, 2, 64, 64, [0, 0], [30, 9], 2)
    wide = i32(np.pad(s.table, ((0, 0), (0, 5)), constant_values=1 << 20))[:, :s.table.shape[1]]
    s.check(s.cache.attend(s.q, wide, i32(s.cu)))


def test_the_same_bits_again():
    s = Setup("mxfp8", 64, 2, 128, 128, [5000, 100, 777], [1, 7, 3], 4)
    first = s.cache.attend(s.q, *s.args())
    for _ in range(3):
        assert torch.equal(first, s.cache.attend(s.q, *s.args()))


def test_offsets_past_32_bits():
    """Vectors whose bytes lie past 4 GiB of a plane."""
    pages, page, heads, dim = 18000, 64, 32, 128
    c = mx.PagedCache(pages, page, heads, dim, dim, mx.FMT_MXFP8)
    g = synth.rng(341)
    kv = [bf16_dev(synth.to_bf16_bits(g.standard_normal((100, heads, dim)))) for _ in range(2)]
    q = bf16_dev(synth.to_bf16_bits(g.standard_normal((1, heads, dim))))
    far, near = i32([[pages - 1, pages - 2]]), i32([[0, 1]])
    got = []
    for table in (far, near):
        c.write(*kv, table, i32([0, 100]))
        got.append(c.attend(q, table, i32([0, 1]), i32([99])))
    assert torch.equal(*got) and got[0].any()


def test_nothing_to_do():
    c = mx.PagedCache(2, 4, 1, 32, 32, mx.FMT_MXFP4)
    z = torch.zeros(0, 2, 32, dtype=torch.bfloat16, device="cuda")
    assert c.attend(z, i32([[0]]), i32([0, 0])).shape == (0, 2, 32)
    assert c.attend(z, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), i32([0])).shape == (0, 2, 32)
    x = torch.ones(3, 2, 32, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 5.0)
    c.attend(x, i32([[0]]), i32([1, 1]), out=out)
    assert bool((out == 5.0).all())
    empty = mx.PagedCache(0, 4, 1, 32, 32, mx.FMT_MXFP4)
    assert not empty.attend(x, i32([[0]]), i32([0, 3])).any()


def test_streams_graphs_and_other_devices(monkeypatch):
    s = Setup("nvfp4", 16, 2, 64, 64, [500, 90], [3, 4], 2)
    table, cu, start = s.args()
    mask = tree_mask(s.g, s.new, s.rows, 0)
    m = torch.from_numpy(mask).cuda()
    want = s.cache.attend(s.q, table, cu, start, tree_mask=m)
    s.check(want, mask)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for st in streams:  # two calls at once
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append([s.cache.attend(s.q, table, cu, start, tree_mask=m) for _ in range(3)])
    for st in streams:
        torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(want, x) for xs in got for x in xs)
    graphs = []
    for _ in range(2):  # two graphs, each with its own workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = s.cache.attend(s.q, table, cu, start, tree_mask=m)
        graphs.append((graph, out))
    for i in range(4):  # new queries, masks and lengths on every replay
        s.q.copy_(bf16_dev(synth.to_bf16_bits(s.g.standard_normal(tuple(s.q.shape)))))
        mask = tree_mask(s.g, s.new, s.rows, 0)
        m.copy_(torch.from_numpy(mask))
        s.have = [500 - 100 * i, 90 - i]
        start.copy_(i32(s.have))
        for graph, out in graphs:
            graph.replay()
            torch.cuda.synchronize()
            s.check(out, mask)
            assert torch.equal(out, s.cache.attend(s.q, table, cu, start, tree_mask=m))
    monkeypatch.setattr(mx.ops, "_current_gpu", lambda: -1)  # as if another device were the current one
    s.check(s.cache.attend(s.q, table, cu, start, tree_mask=m), mask)


def test_refusals():
    c = mx.PagedCache(4, 8, 2, 64, 32, mx.FMT_MXFP4)
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    q, t, cu = z(3, 4, 64), i32([[0]]), i32([0, 3])
    m = z(3, 3, d=torch.bool)
    bad = [lambda: c.attend(q.float(), t, cu), lambda: c.attend(q[:, :3], t, cu), lambda: c.attend(z(3, 0, 64), t, cu),
           lambda: c.attend(z(3, 4, 32), t, cu), lambda: c.attend(q[0], t, cu), lambda: c.attend(q, t.long(), cu),
           lambda: c.attend(q, t, cu[:1]), lambda: c.attend(q, t, cu, i32([0, 0])), lambda: c.attend(q.cpu(), t, cu),
           lambda: c.attend(q, t, cu, tree_mask=m.float()), lambda: c.attend(q, t, cu, tree_mask=m[:2]),
           lambda: c.attend(q, t, cu, tree_mask=m[0]), lambda: c.attend(q, t, cu, tree_mask=m.t()),
           lambda: c.attend(q, t, cu, tree_mask=m[:1].expand(3, 3)), lambda: c.attend(q, t, cu, out=z(3, 4, 64)),
           lambda: c.attend(q, t, cu, out=z(2, 4, 32)), lambda: c.attend(q, t, cu, out=z(3, 4, 32, d=torch.float16)),
           lambda: c.attend(q, t, cu, out_dtype=torch.float16), lambda: c.attend(q.requires_grad_(), t, cu),
           lambda: mx.PagedCache(4, 8, 2, 64, 0, mx.FMT_MXFP4).attend(z(3, 4, 64), t, cu),
           lambda: mx.PagedCache(4, 8, 1, 288, 32, mx.FMT_MXFP4).attend(z(3, 4, 288), t, cu)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
    for scale in (float("nan"), float("inf")):
        with pytest.raises(mx.Mxfp4Error):
            c.attend(z(3, 4, 64), t, cu, scale=scale)
    with pytest.raises(mx.Mxfp4Error):  # rows 8-byte aligned
        c.attend(z(3, 4, 68)[:, :, 4:], t, cu)
    with pytest.raises(mx.Mxfp4Error):  # results on each other
        c.attend(z(3, 4, 64), t, cu, out=z(3, 1, 32).expand(3, 4, 32))
