"""GPU parity of the attention over the paged cache with the float64 oracle where its work is cut up differently: many rows
a key head (tiles of 64, 128 and 256 rows), heads side by side, contexts in few and in many parts, more items than workers.
The tolerance is that of test_gpu_attend.py."""

import numpy as np
import pytest
import torch

import mixed_precision_moe_amd as mx
from mixed_precision_moe_amd import synth
from oracle import attend as A
from tests.gpu_common import bf16_dev, bf16_host_f64
from tests.test_gpu_attend import FMTS, Setup, i32, tolerance, tree_mask

pytestmark = pytest.mark.gpu

# rows a key head: 33 to 64, 65 and more, more than 512, each a whole number of tiles and not
MANY = [([40, 30], 1), ([64], 1), ([21, 12], 5), ([128], 1), ([33, 40, 1], 8), ([130, 7], 2), ([256, 250], 4), ([300], 2)]


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("dims", [(64, 64), (128, 96), (192, 128), (256, 224)])
@pytest.mark.parametrize("new,group", MANY)
def test_many_rows_up_to_their_own_position(fmt, dims, new, group):
    have = [150, 0, 67][:len(new)]
    s = Setup(fmt, 24, 1, *dims, have, new, group, lead=1, tail=2)
    out = torch.full((s.rows, group, dims[1]), 7.0, dtype=torch.bfloat16, device="cuda")
    s.check(s.cache.attend(s.q, *s.args(), out=out), fill=7.0)


@pytest.mark.parametrize("k_dim,v_dim", [(16, 16), (80, 48), (144, 112), (176, 16), (208, 240)])
@pytest.mark.parametrize("new", [[40], [90, 3]])
def test_many_rows_dimensions_of_sixteen(k_dim, v_dim, new):
    s = Setup("nvfp4", 16, 3, k_dim, v_dim, [100, 5][:len(new)], new, 1)
    s.check(s.cache.attend(s.q, *s.args()))


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("new,group", [([50, 9], 1), ([33, 64], 4), ([200], 4)])
def test_many_rows_of_trees(fmt, dims, new, group):
    s = Setup(fmt, 16, 2, *dims, [130, 1][:len(new)], new, group)
    mask = tree_mask(s.g, s.new, s.rows, 0)
    mask[3] = False
    s.check(s.cache.attend(s.q, *s.args(), tree_mask=torch.from_numpy(mask).cuda()), mask)
    none = np.zeros((s.rows, 0), bool)
    s.check(s.cache.attend(s.q, *s.args(), tree_mask=torch.from_numpy(none).cuda()), none)


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("new,group,k_dim", [([40], 1, 64), ([60, 20], 2, 128), ([60], 2, 192), ([60], 2, 256), ([260], 3, 64)])
def test_many_rows_without_pages_and_before_the_first_position(fmt, new, group, k_dim):
    s = Setup(fmt, 4, 2, k_dim, 128 if k_dim == 192 else k_dim, [200, 2][:len(new)], new, group)
    table = s.table.copy()
    table[0, 0], table[0, 3], table[0, 20:45], table[-1, 1] = s.cache.dims.num_pages, -7, np.iinfo(np.int32).max, -1
    s.check(s.cache.attend(s.q, i32(table), *s.args()[1:]), table=table)
    s.check(s.cache.attend(s.q, i32(table[:, :7]), *s.args()[1:]), table=table[:, :7])
    assert not s.cache.attend(s.q, i32(table[:, :0]), *s.args()[1:]).any()
    start = [-9, -50][:len(new)]
    s.check(s.cache.attend(s.q, i32(s.table), i32(s.cu), i32(start)), start=start)
    for scale in (0.0, -0.3):
        s.check(s.cache.attend(s.q, *s.args(), scale=scale), scale=scale)
    empty = mx.PagedCache(0, 4, 2, k_dim, k_dim, FMTS[fmt], *((2.0, 3.0) if fmt == "nvfp4" else ()))
    assert not empty.attend(s.q, *s.args()).any()


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("new,group,k_dim", [([40], 1, 128), ([70], 2, 128), ([70], 2, 192), ([260], 3, 64)])
def test_many_rows_nan_in_hidden_places(fmt, new, group, k_dim):
    """A draft whose keys and values are not numbers reaches those rows alone that see it."""
    s = Setup(fmt, 16, 2, k_dim, 128, [20], new, group)
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    mask = tree_mask(s.g, s.new, s.rows, 0)
    mask[:, 2] = False
    mask[2, 2] = True  # seen by itself alone
    page, slot = s.table[0, 22 // 16], 22 % 16
    for plane in ("k", "v"):
        getattr(s.cache, plane + "_s")[page, slot, 0] = nan
        if fmt == "mxfp8":
            getattr(s.cache, plane + "_q")[page, slot, 1] = 0x7F
    got = s.cache.attend(s.q, *s.args(), tree_mask=torch.from_numpy(mask).cuda())
    rows = [t for t in range(s.rows) if t != 2]
    clean = mask.copy()
    clean[2] = False
    with np.errstate(all="ignore"):
        out, weight, score = A.attend_ref(bf16_host_f64(s.q), *s.values(), s.cu, s.have, s.table, 16, clean)
    tol = tolerance(out, weight, score, k_dim, 20 + new[0], 2.0 ** -8)
    assert np.all(np.abs(got.double().cpu().numpy() - out)[rows] <= tol[rows])
    assert bool(torch.isnan(got[2, :group]).all())


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("heads", [1, 2, 3, 4, 6, 8])
@pytest.mark.parametrize("page,k_dim,v_dim,group", [(64, 128, 128, 4), (32, 64, 64, 20), (24, 128, 96, 3), (10, 192, 64, 18)])
def test_heads_side_by_side(fmt, heads, page, k_dim, v_dim, group):
    """Few rows, contexts longer than a unit; pages of whole tiles and others."""
    s = Setup(fmt, page, heads, k_dim, v_dim, [300, 31, 0, 129], [1, 1, 1, 1], group)
    s.check(s.cache.attend(s.q, *s.args()))


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("new,group,k_dim,have", [(1, 2, 64, 20000), (4, 8, 128, 9000), (50, 1, 64, 9000), (40, 2, 192, 7000),
                                                  (40, 2, 256, 3000), (140, 4, 64, 4000)])
def test_one_context_in_many_parts(fmt, new, group, k_dim, have):
    s = Setup(fmt, 64, 1, k_dim, 128 if k_dim == 192 else k_dim, [have], [new], group)
    s.check(s.cache.attend(s.q, *s.args()))
    s.check(s.cache.attend(s.q, *s.args(), out_dtype=torch.float32), half_step=2.0 ** -24)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_more_items_than_workers(fmt):
    g = np.random.default_rng(8)
    have, new = [int(x) for x in g.integers(0, 200, 130)], [1 + int(x) for x in g.integers(0, 2, 130)]
    s = Setup(fmt, 16, 32, 32, 32, have, new, 2)
    s.check(s.cache.attend(s.q, *s.args()))
    mask = tree_mask(s.g, new, s.rows, 0)
    s.check(s.cache.attend(s.q, *s.args(), tree_mask=torch.from_numpy(mask).cuda()), mask)


def test_many_rows_the_same_bits_again_and_captured():
    s = Setup("mxfp8", 64, 2, 128, 128, [900, 100], [140, 7], 4)
    args = s.args()
    first = s.cache.attend(s.q, *args)
    s.check(first)
    assert torch.equal(first, s.cache.attend(s.q, *args))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.cache.attend(s.q, *args)
    for i in range(3):
        s.q.copy_(bf16_dev(synth.to_bf16_bits(s.g.standard_normal(tuple(s.q.shape)))))
        s.have = [900 - 333 * i, 100 - i]
        args[2].copy_(i32(s.have))
        graph.replay()
        torch.cuda.synchronize()
        s.check(out)
        assert torch.equal(out, s.cache.attend(s.q, *args))
