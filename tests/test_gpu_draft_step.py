"""Drafted decoding as a serving program runs it: queries and keys are turned by their positions, keys and values written into
the cache through the pool's page table, the tree of drafts attends over it, the accepted branch is moved together, the pages
of the rest go back; two samples continue from one sequence.  At every step the result is what a cache holds that was written
token by token."""

import numpy as np
import pytest
import torch

import mixed_precision_moe_amd as mx
from mixed_precision_moe_amd import synth
from oracle import attend as A
from oracle import cache as C
from oracle import rotary as R
from tests.gpu_common import bf16_dev, bf16_host_bits, bf16_host_f64
from tests.test_gpu_attend import GS, FMTS, i32, tolerance, tree_mask

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", list(FMTS))
def test_drafted_decoding(fmt):
    g = synth.rng(370)
    B, heads, group, dim, v_dim, page, W = 3, 2, 3, 64, 32, 4, 6
    cache = mx.PagedCache(60, page, heads, dim, v_dim, FMTS[fmt], *GS[fmt])
    pool = mx.PagePool(cache)
    table = torch.full((2 * B, 14), -1, dtype=torch.int32, device="cuda")
    rot = mx.Rotary(32, offset=16, scaling=dict(kind="linear", factor=2.0))
    turns = rot._turns.cpu().numpy()
    kept = [[] for _ in range(2 * B)]  # accepted (key, value) bits of each row, as turned
    lengths = np.zeros(2 * B, np.int64)

    def step(rows, new, accept):
        """Drafts of the given rows; `accept` of each are kept."""
        cu = np.concatenate([[0], np.cumsum(new)])
        mask = tree_mask(g, new, int(cu[-1]), 0, W)
        depth = mask.sum(1) - 1  # a draft's position is its depth in the tree
        positions = np.concatenate([[lengths[r] + d for d in depth[cu[i]:cu[i + 1]]] for i, r in enumerate(rows)])
        q, k = (synth.to_bf16_bits(g.standard_normal((int(cu[-1]), h, dim))) for h in (heads * group, heads))
        v = synth.to_bf16_bits(g.standard_normal((int(cu[-1]), heads, v_dim)))
        room = lengths.copy()
        room[rows] += new
        assert int(pool.resize(table, i32(room))) == 0
        at = table[torch.tensor(rows, device="cuda")].contiguous()
        start = i32(lengths[rows])
        qt, kt = rot(bf16_dev(q), bf16_dev(k), i32(positions))
        for x, y in ((q, qt), (k, kt)):
            x64 = bf16_host_f64(bf16_dev(x))
            want = R.rotary_ref(x64, positions, turns, 16)
            assert np.all(np.abs(bf16_host_f64(y) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.abs(x64).max())
        cache.write(kt, bf16_dev(v), at, i32(cu), start)
        out = cache.attend(qt, at, i32(cu), start, tree_mask=torch.from_numpy(mask).cuda())
        # against a contiguous cache of what was kept and the drafts
        kb = bf16_host_bits(kt)
        for i, r in enumerate(rows):
            seq = kept[r] + [(kb[t], v[t]) for t in range(cu[i], cu[i + 1])]
            held = [C.decode_ref(*C.encode_ref(np.stack([s[p] for s in seq]), fmt, GS[fmt][p]), fmt, GS[fmt][p]) for p in range(2)]
            mine = slice(cu[i], cu[i + 1])
            want = A.attend_ref(bf16_host_f64(qt)[mine], *held, [0, new[i]], [int(lengths[r])], [list(range(len(seq)))], 1, mask[mine])
            tol = tolerance(*want, dim, len(seq), 2.0 ** -8)
            assert np.all(np.abs(bf16_host_f64(out)[mine] - want[0]) <= tol)
        # a branch: one draft and its ancestors
        path = np.full((len(rows), W), -1, np.int32)
        for i, r in enumerate(rows):
            leaf = int(np.argmin(np.abs(depth[cu[i]:cu[i + 1]] + 1 - accept)))
            branch = np.flatnonzero(mask[cu[i] + leaf])
            path[i, :len(branch)] = branch
            kept[r] += [(kb[cu[i] + j], v[cu[i] + j]) for j in branch]
            lengths[r] += len(branch)
        assert cache.compact(at, start, i32(path)).tolist() == list(lengths[rows])
        assert int(pool.resize(table, i32(lengths))) == 0

    def check():
        every = [r for r in range(2 * B) if lengths[r]]
        cu = np.concatenate([[0], np.cumsum(lengths[every])])
        got = cache.read(table[torch.tensor(every, device="cuda")].contiguous(), i32(cu), rows=int(cu[-1]))
        for p in range(2):
            held = np.stack([s[p] for r in every for s in kept[r]])
            np.testing.assert_array_equal(bf16_host_bits(got[p]), C.bf16_bits(C.decode_ref(*C.encode_ref(held, fmt, GS[fmt][p]), fmt, GS[fmt][p])))
        used = set(table[table >= 0].tolist())
        assert int((pool.refs > 0).sum()) == len(used)

    step([0, 1, 2], [5, 1, 6], 3)
    check()
    step([0, 1, 2], [6, 6, 2], 2)
    check()
    src, dst = [0, 0, 2], [3, 4, 5]
    at = [int(lengths[0]), int(lengths[0]) - 1, int(lengths[2])]
    assert int(pool.fork(table, i32(src), i32(dst), i32(at))) == 0
    for s, d, n in zip(src, dst, at):
        kept[d], lengths[d] = kept[s][:n], n
    check()
    step([0, 3, 4, 5], [4, 6, 3, 1], 3)  # samples go their own ways
    check()
    step([1, 2, 3, 5], [2, 6, 6, 6], 4)
    check()
    pool.resize(table, i32([0] * (2 * B)))
    assert not pool.refs.any() and bool((table == -1).all())


def test_a_captured_step():
    """Rotary, write, attention, compaction and the pool in one graph, on lengths that the graph itself moves on."""
    g = synth.rng(371)
    B, heads, group, dim, page, n = 2, 2, 2, 64, 8, 4
    cache = mx.PagedCache(40, page, heads, dim, dim, mx.FMT_MXFP8)
    twin = mx.PagedCache(40, page, heads, dim, dim, mx.FMT_MXFP8)
    rot = mx.Rotary(dim)
    mask = torch.from_numpy(tree_mask(g, [n] * B, B * n, 0)).cuda()
    cu = i32([0, n, 2 * n])
    draft = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B)

    def state(c):
        return c, mx.PagePool(c), torch.full((B, 12), -1, dtype=torch.int32, device="cuda"), i32([0, 0])

    def run(c, pool, table, lengths, q, k, v, path):
        missing = pool.resize(table, lengths + n)
        qt, kt = rot(q, k, lengths.repeat_interleave(n) + draft)
        c.write(kt, v, table, cu, lengths)
        out = c.attend(qt, table, cu, lengths, tree_mask=mask)
        lengths.copy_(c.compact(table, lengths, path))
        pool.resize(table, lengths)
        return out, missing

    new = lambda: (bf16_dev(synth.to_bf16_bits(g.standard_normal((B * n, h, dim)))) for h in (heads * group, heads, heads))  # noqa: E731
    q, k, v = new()
    path = i32([[0, 2, -1, -1], [0, 1, 3, -1]])
    mine, eager = state(cache), state(twin)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(*mine, q, k, v, path)
    torch.cuda.current_stream().wait_stream(s)
    run(*eager, q, k, v, path)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, missing = run(*mine, q, k, v, path)
    for i in range(4):
        for t, x in zip((q, k, v), new()):
            t.copy_(x)
        path.copy_(i32([[0, 1 + i % 3, -1, -1], [0, 1, 2, 3 if i % 2 else -1]]))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = run(*eager, q, k, v, path)
        assert torch.equal(out, want) and int(missing) == 0 and torch.equal(mine[2], eager[2]) and torch.equal(mine[3], eager[3])
        used = mine[2][mine[2] >= 0].long()
        for name in ("k_q", "k_s", "v_q", "v_s"):
            assert torch.equal(getattr(cache, name)[used], getattr(twin, name)[used])
