"""GPU parity of compaction, page copies and the page pool with the plain oracle: every byte and every number."""

import numpy as np
import pytest
import torch

import mixed_precision_moe_amd as mx
from mixed_precision_moe_amd import synth
from oracle import pages as P

pytestmark = pytest.mark.gpu
FMTS = {"mxfp4": mx.FMT_MXFP4, "nvfp4": mx.FMT_NVFP4, "mxfp8": mx.FMT_MXFP8}


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def make(fmt, pages, page, heads, k_dim, v_dim, seed=0, odd=False):
    """A cache of arbitrary bytes, and its planes as the oracle holds them; odd: scales on odd addresses."""
    g = synth.rng(360, seed, pages, page)
    by, block = (1 if fmt == "mxfp8" else 2), (16 if fmt == "nvfp4" else 32)
    store = []
    for d in (k_dim // by, k_dim // block, v_dim // by, v_dim // block):
        a = g.integers(0, 256, (pages, page, heads, d), dtype=np.uint8)
        if d == 0:
            store.append(None)
            continue
        pad = 1 if odd and len(store) % 2 else 0
        flat = torch.zeros(a.size + pad, dtype=torch.uint8, device="cuda")
        flat[pad:] = torch.from_numpy(a.reshape(-1)).cuda()
        store.append(flat[pad:].view(a.shape))
    c = mx.PagedCache(pages, page, heads, k_dim, v_dim, FMTS[fmt], storage=store)
    planes = [t.cpu().numpy().reshape(pages * page, -1).copy() for t in store if t is not None]
    return c, planes, g


def same(c, planes):
    for t, a in zip((t for t in (c.k_q, c.k_s, c.v_q, c.v_s) if t is not None), planes):
        np.testing.assert_array_equal(t.cpu().numpy().reshape(a.shape), a)


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("page,heads,k_dim,v_dim,B,W", [
    (16, 2, 64, 64, 1, 1), (1, 1, 32, 32, 3, 5), (24, 8, 192, 128, 5, 64), (64, 3, 96, 160, 4, 9), (7, 5, 32, 0, 6, 33),
    (5, 1, 576, 0, 2, 700), (3, 1, 32, 32, 40, 300), (128, 16, 256, 224, 2, 40)])
def test_compaction(fmt, page, heads, k_dim, v_dim, B, W):
    print(f"compact {fmt} page={page} heads={heads} dims={k_dim},{v_dim} B={B} W={W}", flush=True)
    start = np.random.default_rng(W).integers(0, 2 * page + 1, B)
    need = [-(-(int(s) + W) // page) for s in start]
    c, planes, g = make(fmt, sum(need) + 1, page, heads, k_dim, v_dim, odd=heads == 3)
    order = list(g.permutation(sum(need) + 1))
    table = np.full((B, max(need)), -1, np.int32)
    for b, n in enumerate(need):
        table[b, :n] = [order.pop() for _ in range(n)]
    path = np.full((B, W + 3), -1, np.int32)
    for b in range(B):
        n = [0, 1, W, W // 2][b % 4] if b else W - 1
        chosen = np.sort(g.permutation(W)[:n])
        path[b, :n] = chosen
        if b % 3 == 1:  # ends with what does not increase
            path[b, n:] = path[b, n - 1] if n else -3
    want = P.compact_ref(planes, table, start, path, page, c.dims.num_pages)
    wide = torch.full((B, W + 9), 5, dtype=torch.int32, device="cuda")
    wide[:, :W + 3] = i32(path)
    lengths = c.compact(i32(table), i32(start), wide[:, :W + 3])
    same(c, planes)
    assert lengths.tolist() == want


def test_compaction_without_pages_and_without_drafts():
    c, planes, g = make("mxfp8", 6, 4, 2, 32, 32)
    table = np.array([[0, 9, 1], [-1, 2, 3], [5, -4, 4]], np.int32)
    start, path = [2, 1, 0], [[1, 3, 5, 7], [3, 4, 6, 8], [0, 1, 9, 11]]
    want = P.compact_ref(planes, table, start, path, 4, 6)
    assert c.compact(i32(table), i32(start), i32(path)).tolist() == want == [6, 5, 4]
    same(c, planes)
    assert c.compact(i32(table), i32([-3, 1 << 30, 100]), i32(path)).tolist() == [1, (1 << 30) + 4, 104]
    c.compact(i32(table[:, :0]), i32(start), i32(path))
    P.compact_ref(planes, table, [-3, 1 << 30, 100], path, 4, 6)
    same(c, planes)
    assert c.compact(i32(table), i32(start), torch.zeros(3, 0, dtype=torch.int32, device="cuda")).tolist() == start
    assert c.compact(torch.zeros(0, 3, dtype=torch.int32, device="cuda"), i32([]), torch.zeros(0, 2, dtype=torch.int32, device="cuda")).shape == (0,)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_page_copies(fmt):
    c, planes, g = make(fmt, 40, 24, 3, 96, 64, odd=True)
    src, dst = [3, 4, 40, -1, 5, 7, 3], [10, 11, 12, 13, 14, 15, 16]
    rows = [24, 1, 5, 5, 0, 23, 99]
    for s, d, r in zip(src, dst, rows):
        if 0 <= s < 40:
            for a in planes:
                a[d * 24:d * 24 + min(r, 24)] = a[s * 24:s * 24 + min(r, 24)]
    c.copy_pages(i32(src), i32(dst), i32(rows))
    same(c, planes)
    c.copy_pages(i32([0, 1]), i32([20, 21]))
    for a in planes:
        a[20 * 24:22 * 24] = a[:48]
    same(c, planes)
    c.copy_pages(i32([]), i32([]))
    same(c, planes)


class Pool:
    """A pool over caches, and what the oracle holds of it."""

    def __init__(self, pages, page, rows, columns, caches=1, fmt="mxfp8", seed=0):
        made = [make(fmt, pages, page, 2, 32, 64, seed + i) for i in range(caches)]
        self.page, self.g = page, made[0][2]
        self.caches, self.planes = [m[0] for m in made], [m[1] for m in made]
        self.pool = mx.PagePool(*self.caches)
        self.table, self.refs = np.full((rows, columns), -1, np.int32), np.zeros(pages, np.int32)
        self.wide = torch.full((rows, columns + 3), 77, dtype=torch.int32, device="cuda")
        self.dev = self.wide[:, :columns]
        self.dev.fill_(-1)

    def all_planes(self):
        return [a for planes in self.planes for a in planes]

    def check(self, missing, want):
        assert missing.shape == () and int(missing) == want
        np.testing.assert_array_equal(self.dev.cpu().numpy(), self.table)
        np.testing.assert_array_equal(self.pool.refs.cpu().numpy(), self.refs)
        assert bool((self.wide[:, self.table.shape[1]:] == 77).all())
        for c, planes in zip(self.caches, self.planes):
            same(c, planes)

    def resize(self, lengths):
        want = P.resize_ref(self.refs, self.table, lengths, self.page, self.all_planes())
        self.check(self.pool.resize(self.dev, i32(lengths)), want)
        return want

    def fork(self, src, dst, lengths):
        want = P.fork_ref(self.refs, self.table, src, dst, lengths, self.page, self.all_planes())
        self.check(self.pool.fork(self.dev, i32(src), i32(dst), i32(lengths)), want)
        return want


@pytest.mark.parametrize("pages,page,rows,columns", [(60, 4, 6, 12), (9, 1, 3, 20), (20000, 16, 70, 130), (300, 24, 1, 200),
                                                     (3000, 2, 1500, 5), (1, 8, 2, 2)])
def test_a_pool_through_many_steps(pages, page, rows, columns):
    print(f"pool pages={pages} page={page} rows={rows} columns={columns}", flush=True)
    p = Pool(pages, page, rows, columns, caches=2 if rows < 100 else 1)
    g = np.random.default_rng(pages)
    lengths, short = np.zeros(rows, int), 0
    for step in range(6):
        grown = lengths + g.integers(0, 3 * page + 1, rows)
        if step == 3:
            grown[g.random(rows) < 0.4] = 0
        grown = np.where(g.random(rows) < 0.2, -1, grown)  # left alone
        short += p.resize(grown)
        lengths = np.where(grown < 0, lengths, grown)
        held = np.array([P.held_ref(r, pages) * page for r in p.table])
        lengths = np.minimum(lengths, held)
        if rows > 1:
            order = g.permutation(rows)
            n = max(1, rows // 3)
            dst, src = order[:n], g.choice(order[n:], n)
            at = np.array([g.integers(0, lengths[s] + 1) for s in src])
            short += p.fork(src, dst, at)
            lengths[dst] = np.minimum(at, [P.held_ref(p.table[d], pages) * page for d in dst])
        back = np.maximum(0, lengths - g.integers(0, 2 * page, rows))  # into shared pages too
        short += p.resize(back)
        lengths = np.minimum(back, [P.held_ref(r, pages) * page for r in p.table])
    assert short > 0 or pages > 20  # the smallest pools run out
    assert p.resize(np.zeros(rows, int)) == 0
    assert not p.refs.any() and (p.table == -1).all()


def test_shared_pages_are_replaced_where_a_length_ends_in_them():
    p = Pool(20, 4, 4, 6)
    p.resize([10, 0, 0, 0])
    p.fork([0, 0], [1, 2], [10, 8])
    assert p.refs[p.table[0, 0]] == 3 and p.refs[p.table[0, 2]] == 1
    p.resize([10, 6, 8, -1])  # row 1 ends inside a page that three rows hold
    assert p.table[1, 1] != p.table[0, 1] and p.refs[p.table[0, 1]] == 2
    p.resize([7, -1, 7, -1])  # both of those that share it end inside it: two copies, the page is free
    assert p.table[0, 1] != p.table[2, 1]
    p.resize([0, 0, 0, 0])


def test_pairs_that_are_passed_over():
    p = Pool(30, 4, 6, 5)
    p.resize([9, 5, 3, 7, 0, 0])
    p.fork([0, 1, 0, 6, 0, -1, 2, 2, 0], [4, 4, 6, 5, -1, 5, 5, 0, 3], [9, 5, 9, 9, 9, 9, 2, 3, -1])
    p.fork([0, 3], [5, 3], [20, 7])  # longer than what the row holds; a row onto itself
    p.fork([], [], [])
    p.resize([1 << 30, -5, 4, 4, 0, 21])  # more than the table holds


def test_tables_with_holes():
    p = Pool(30, 4, 4, 6)
    p.table[:] = [[1, 2, 99, 3, -1, -1], [-7, 4, 5, -1, -1, -1], [6, 7, 8, 30, 30, 9], [-1] * 6]
    p.dev.copy_(i32(p.table))
    for page in (1, 2, 6, 7, 8):
        p.refs[page] = 1
    p.pool.refs.copy_(i32(p.refs))
    p.fork([0, 2], [3, 1], [14, 9])
    p.resize([12, 20, 4, 0])


def test_no_pages_no_rows_no_columns():
    p = Pool(5, 4, 2, 3)
    assert int(p.pool.resize(p.dev[:0], i32([]))) == 0
    assert int(p.pool.resize(p.dev[:, :0], i32([3, 4]))) == 0
    none = mx.PagePool(mx.PagedCache(0, 4, 1, 32, 32))
    t = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    assert int(none.resize(t, i32([5, 2]))) == 3 and bool((t == -1).all())


def test_streams_graphs_and_other_devices(monkeypatch):
    """A step that is captured: trim to what was accepted, make room for the next drafts."""
    p = Pool(400, 16, 8, 20)
    lengths, room = i32([0] * 8), i32([0] * 8)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.pool.resize(p.dev, lengths)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        p.pool.resize(p.dev, lengths)
        missing = p.pool.resize(p.dev, room)
    g = np.random.default_rng(3)
    have = np.zeros(8, int)
    for i in range(5):
        have = have + g.integers(0, 40, 8)
        lengths.copy_(i32(have))
        room.copy_(i32(have + 33))
        graph.replay()
        torch.cuda.synchronize()
        P.resize_ref(p.refs, p.table, have, 16, p.all_planes())
        p.check(missing, P.resize_ref(p.refs, p.table, have + 33, 16, p.all_planes()))
        p.fork([0], [7], [int(have[0])])  # eager, between the replays
        have[7] = have[0]
    monkeypatch.setattr(mx.ops, "_current_gpu", lambda: -1)  # as if another device were the current one
    p.resize([5] * 8)
    c, planes, g = make("mxfp4", 4, 8, 2, 32, 32)
    want = P.compact_ref(planes, [[2, 1]], [3], [[1, 4]], 8, 4)
    assert c.compact(i32([[2, 1]]), i32([3]), i32([[1, 4]])).tolist() == want
    same(c, planes)


def test_offsets_past_32_bits():
    """Rows whose bytes lie past 4 GiB of a plane."""
    pages, page, heads, dim = 18000, 64, 32, 128
    c = mx.PagedCache(pages, page, heads, dim, 0, mx.FMT_MXFP8)
    g = synth.rng(361)
    bits = torch.from_numpy(g.integers(0, 256, (page, heads, dim), dtype=np.uint8)).cuda()
    c.k_q[pages - 1] = bits
    c.copy_pages(i32([pages - 1]), i32([pages - 3]), i32([40]))
    assert torch.equal(c.k_q[pages - 3, :40], bits[:40]) and not c.k_q[pages - 3, 40:].any()
    c.compact(i32([[pages - 1, pages - 3]]), i32([60]), i32([[6]]))  # from the second page into the first
    assert torch.equal(c.k_q[pages - 1, 60], bits[2]) and torch.equal(c.k_q[pages - 1, :60], bits[:60])


def test_refusals():
    c = mx.PagedCache(4, 8, 2, 64, 32, mx.FMT_MXFP4)
    other = mx.PagedCache(5, 8, 2, 64, 32, mx.FMT_MXFP4)
    pool = mx.PagePool(c)
    t, n, path = i32([[0, 1], [2, -1]]), i32([3, 4]), i32([[0, 1], [0, 2]])
    bad = [lambda: c.compact(t.long(), n, path), lambda: c.compact(t, n[:1], path), lambda: c.compact(t, n, path[:1]),
           lambda: c.compact(t, n, path.t()), lambda: c.compact(t, n, path.long()), lambda: c.compact(t.cpu(), n, path),
           lambda: c.copy_pages(n, n[:1]), lambda: c.copy_pages(n.long(), n), lambda: c.copy_pages(t, n), lambda: c.copy_pages(n, n, t),
           lambda: pool.resize(t, n[:1]), lambda: pool.resize(t, n.long()), lambda: pool.resize(t[0], n), lambda: pool.resize(t, n.cpu()),
           lambda: pool.resize(t[:1].expand(2, 2), n), lambda: pool.fork(t, n, n[:1], n), lambda: pool.fork(t, n, n, n.float()),
           lambda: mx.PagePool(), lambda: mx.PagePool(c, other), lambda: mx.PagePool(c, refs=n), lambda: mx.PagePool(n),
           lambda: mx.PagePool(c, refs=torch.zeros(4, dtype=torch.int32))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(mx.Mxfp4Error):
        pool.fork(t, *(torch.zeros(70000, dtype=torch.int32, device="cuda") for _ in range(3)))
