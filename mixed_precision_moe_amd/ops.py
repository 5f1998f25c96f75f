"""The balance loss, the 4-bit matrix-vector products, the block-quantized paged cache with the attention over it and
its page pool: the torch binding of their C entry points.  Like the rest of the binding it checks dtypes, shapes and devices, allocates
outputs and passes raw pointers; the work runs on the current stream of the tensors' device."""

import ctypes
import functools

import torch

from . import _lib
from ._lib import CacheDims, check

FMT_MXFP4 = 0  # E2M1, an E8M0 scale per 32 elements (quantize)
FMT_NVFP4 = 1  # E2M1, an E4M3 scale per 16 elements and a global scale (nvfp4_quantize)
FMT_MXFP8 = 2  # E4M3, an E8M0 scale per 32 elements (the cache only)

_GROUP = {FMT_MXFP4: 32, FMT_NVFP4: 16, FMT_MXFP8: 32}


# The stream's handle without the object around it: about 2 us of a call that a small kernel does not hide.
_stream_of = torch._C._cuda_getCurrentRawStream


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _need_int32(*sizes):
    """ctypes would pass the low 32 bits of a larger number on."""
    for n in sizes:
        if not -1 << 31 <= n < 1 << 31:
            raise ValueError(f"a size of {n} does not fit the entry points' 32 bits")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _gpu_of(name, first, *others):
    """The number of the GPU that holds `first` (called `name`) and every other tensor."""
    index = first.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"every tensor must be on {name}'s device")
    return index


_current_gpu = torch.cuda.current_device

# For tensors of the caller's that a kernel has written: a backward pass that saved one must not go on with what it holds now.
_changed = torch.autograd.graph.increment_version


def _check_given(*tensors):
    """Results that the caller gives: what they held before has no gradient through the call."""
    _need(not (torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)),
          "a result that is given must not ask for a gradient")


def _no_tangent(what, *tensors):
    """Refuses forward-mode derivatives, which a kernel behind raw pointers would drop without a word."""
    # outside every dual level, where unpacking would cost a small call more than a microsecond, there are none
    if _forward_ad._current_level >= 0 and any(_forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise ValueError(f"{what} has no forward-mode derivative")


_forward_ad = torch.autograd.forward_ad


def _call(index, fn, *args):
    """fn(*args, stream) on the current stream of GPU `index`, which need not be the current device."""
    if index == _current_gpu():
        status = getattr(_lib.lib(), fn)(*args, _stream_of(index))
    else:
        with torch.cuda.device(index):
            status = getattr(_lib.lib(), fn)(*args, _stream_of(index))
    if status:
        check(fn, status)


# ------------------------------------------------------------------------------------------------
# Balance loss.


def _check_logits(logits):
    """(tokens, experts, elements from row to row; the stride of a single row says nothing)."""
    if logits.dtype != torch.float32 or logits.dim() != 2:
        raise ValueError("logits: fp32 [T, E]")
    T, E = logits.shape
    step, unit = logits.stride()
    if unit != 1 and E > 1:
        raise ValueError("logits' last dimension must be contiguous")
    if T <= 1:
        return T, E, E
    if step < E:
        raise ValueError("logits' rows must not overlap")
    return T, E, step


def _check_mask(mask, T):
    _need(mask.dtype in (torch.bool, torch.uint8) and mask.shape == (T,) and mask.is_contiguous(),
          "token_mask: contiguous bool or uint8 [T]")


@functools.lru_cache(maxsize=256)
def _balance_workspace(T, E):
    return _lib.lib().moe_balance_workspace_bytes(T, E)


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk_ids, mask, T, E, step):
        dev, index = logits.device, logits.get_device()
        nws = _balance_workspace(T, E)
        if nws == 0:
            raise ValueError("invalid balance loss arguments")
        ws = torch.empty(nws, dtype=torch.uint8, device=dev)
        coef, loss = logits.new_empty(E), logits.new_empty(())
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        _call(index, "moe_balance_forward", logits.data_ptr(), T, E, step, topk_ids.data_ptr(), topk_ids.shape[1],
              _ptr(mask), loss.data_ptr(), counts.data_ptr(), coef.data_ptr(), ws.data_ptr(), nws)
        ctx.save_for_backward(logits, mask)
        # d_e, which is neither an input nor an output and which saved-tensor hooks therefore need not see
        ctx.coef, ctx.sizes, ctx.index = coef, (T, E), index
        ctx.mark_non_differentiable(counts)
        ctx.set_materialize_grads(False)
        return loss, counts

    @staticmethod
    def backward(ctx, g, _):
        if torch.is_grad_enabled():
            raise RuntimeError("balance_loss has no second derivative (create_graph)")
        if g is None:
            return None, None, None, None, None, None
        # saved-tensor hooks may return others than were saved: with other strides, which the kernel can take, or unfit
        logits, mask = ctx.saved_tensors
        T, E, step = _check_logits(logits)
        index = ctx.index
        if (T, E) != ctx.sizes or logits.get_device() != index or mask is not None and mask.get_device() != index:
            raise ValueError("the tensors saved for the backward pass have changed")
        if mask is not None:
            _check_mask(mask, T)
        grad = logits.new_empty((T, E))
        _call(index, "moe_balance_backward", logits.data_ptr(), T, E, step, _ptr(mask), ctx.coef.data_ptr(), g.data_ptr(),
              grad.data_ptr())
        return grad, None, None, None, None, None


def balance_loss(logits, topk_ids, token_mask=None):
    """The router's balance loss and per-expert counts.

    logits fp32 [T, E] (rows may be strided), topk_ids int32 [T, k] as `route` returns them (an id outside
    [0, E) is a dropped pair), token_mask bool or uint8 [T] or None: tokens that count.  Returns (loss, counts):
    loss fp32, 0-dim, differentiable in the logits: E / (k V^2) * sum_e counts_e * sum_t softmax(logits_t)_e
    over the V tokens that count (0 without any); counts int32 [E], constants of the gradient.  To capture its backward
    pass into a graph, drop every eager autograd graph of the same leaves first, as torch asks for any backward pass."""
    _gpu_of("logits", logits, topk_ids, token_mask)
    T, E, step = _check_logits(logits)
    _need_int32(E)
    _need(topk_ids.dtype == torch.int32 and topk_ids.dim() == 2 and topk_ids.shape[0] == T and topk_ids.is_contiguous(),
          "topk_ids: contiguous int32 [T, k]")
    _need_int32(topk_ids.shape[1])
    if token_mask is not None:
        _check_mask(token_mask, T)
    return _BalanceLoss.apply(logits, topk_ids, token_mask, T, E, step)


# ------------------------------------------------------------------------------------------------
# Matrix-vector products.


def _check_weights(w_q, w_s, fmt, dims):
    """The shape of the codes, with K in place of K/2."""
    _need(fmt == FMT_MXFP4 or fmt == FMT_NVFP4, "fmt must be FMT_MXFP4 or FMT_NVFP4")
    for t in (w_q, w_s):
        if t.dtype != torch.uint8 or t.dim() != dims or not t.is_contiguous():
            raise ValueError(f"w_q and w_s must be contiguous uint8 {dims}-D")
    *rows, half = w_q.shape
    group = _GROUP[fmt] // 2
    _need(half % group == 0 and list(w_s.shape) == [*rows, half // group], "w_s shape")
    return *rows, 2 * half


def _check_bias(bias, shape):
    """Whether the bias is fp32."""
    if bias is None:
        return 0
    _need((bias.dtype == torch.float32 or bias.dtype == torch.bfloat16) and bias.shape == shape and bias.is_contiguous(),
          "bias: contiguous fp32 or bf16, one value for each row of the weights")
    return 1 if bias.dtype == torch.float32 else 0


def _check_out(out_dtype):
    if out_dtype == torch.bfloat16:
        return 0
    _need(out_dtype == torch.float32, "out_dtype must be bfloat16 or float32")
    return 1


def _check_rows(x, K):
    """(rows, elements from row to row; the stride of a single row says nothing)."""
    _need(x.dtype == torch.bfloat16 and x.dim() == 2 and x.shape[1] == K and x.stride(1) == 1, "x: bf16 rows [*, K]")
    M = x.shape[0]
    if M <= 1:
        return M, K + -K % 8
    ldx = x.stride(0)
    _need(ldx >= K, "x's rows must not overlap")
    return M, ldx


def fp4_matvec(x, w_q, w_s, bias=None, *, fmt=FMT_MXFP4, global_scale=None, out_dtype=torch.bfloat16):
    """y = x W^T (/ global_scale) + b for one or a few rows of x: the decoding form of the W4A16 linear layer,
    on weights as `quantize` (FMT_MXFP4) or `nvfp4_quantize` (FMT_NVFP4, with its global_scale) returns them.

    x bf16 [M, K] (rows may be strided, by a multiple of 8 elements; they and w_q start on 16 bytes), w_q uint8
    [N, K/2], w_s uint8 flat scales [N, K/32] or [N, K/16], bias fp32 or bf16 [N] or None.  Returns y [M, N] in
    out_dtype (bfloat16 or float32)."""
    gpu = _gpu_of("x", x, w_q, w_s, bias)
    N, K = _check_weights(w_q, w_s, fmt, 2)
    M, ldx = _check_rows(x, K)
    _need((global_scale is not None) == (fmt == FMT_NVFP4), "global_scale goes with FMT_NVFP4, and only with it")
    is_fp32 = _check_bias(bias, (N,))
    out_fp32 = _check_out(out_dtype)
    y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _call(gpu, "fp4_matvec", fmt, w_q.data_ptr(), w_s.data_ptr(), 1.0 if global_scale is None else global_scale, N, K,
          _ptr(bias), is_fp32, x.data_ptr(), M, ldx, y.data_ptr(), N, out_fp32)
    return y


def fp4_expert_matvec(x, w_q, w_s, expert_offsets, sorted_pairs, bias=None, *, fmt=FMT_MXFP4, global_scales=None,
                      top_k=1, swiglu=False, out_dtype=torch.bfloat16, y=None):
    """Every routed pair's product with its expert's matrix, on weights in the standard layout.

    x bf16 [P / top_k, K], laid out as for `fp4_matvec`: row p // top_k is the input of pair p (top_k as routed for
    the first product, 1 where every pair has its own row).  w_q uint8 [E, N, K/2], w_s uint8 [E, N, K/32] (NVFP4:
    [E, N, K/16]), bias [E, N] or None, global_scales fp32 [E] (NVFP4).  expert_offsets int32 [E + 1] and
    sorted_pairs int32 [P] as `route` returns them.  Returns y [P, N], or [P, N/2] = silu(gate rows) * up rows with
    swiglu (rows [w1; w3]).  A pair that sorted_pairs does not list keeps what its row of `y` held (without `y` the
    row is undefined)."""
    gpu = _gpu_of("x", x, w_q, w_s, bias, expert_offsets, sorted_pairs, global_scales, y)
    E, N, K = _check_weights(w_q, w_s, fmt, 3)
    M, ldx = _check_rows(x, K)
    for t in (expert_offsets, sorted_pairs):
        _need(t.dtype == torch.int32 and t.dim() == 1 and t.is_contiguous(),
              "expert_offsets and sorted_pairs: contiguous int32 1-D")
    _need_int32(E, top_k)
    _need(expert_offsets.shape[0] == E + 1, "expert_offsets: E + 1 entries")
    P = sorted_pairs.shape[0]
    _need(top_k >= 1 and M * top_k == P, "x must have one row for every top_k pairs")
    _need((global_scales is not None) == (fmt == FMT_NVFP4), "global_scales goes with FMT_NVFP4, and only with it")
    if global_scales is not None:
        _need(global_scales.dtype == torch.float32 and global_scales.shape == (E,) and global_scales.is_contiguous(),
              "global_scales: contiguous fp32 [E]")
    _need(not swiglu or N % 2 == 0, "swiglu needs an even number of rows")
    is_fp32 = _check_bias(bias, (E, N))
    width = N // 2 if swiglu else N
    given = y is not None
    if not given:
        out_fp32 = _check_out(out_dtype)
        y = torch.empty((P, width), dtype=out_dtype, device=x.device)
    else:
        out_fp32 = _check_out(y.dtype)
        _check_given(y)
        _need(y.shape == (P, width) and y.is_contiguous(), "y: contiguous [P, N] (swiglu: [P, N/2])")
    _call(gpu, "fp4_expert_matvec", fmt, w_q.data_ptr(), w_s.data_ptr(), _ptr(global_scales), E, N, K, _ptr(bias),
          is_fp32, x.data_ptr(), ldx, top_k, expert_offsets.data_ptr(), sorted_pairs.data_ptr(), P, 1 if swiglu else 0,
          y.data_ptr(), out_fp32)
    if given:
        _changed(y)
    return y


# ------------------------------------------------------------------------------------------------
# Paged cache.


@functools.lru_cache(maxsize=1024)
def _attend_workspace(fmt, heads, k_dim, v_dim, q_heads, rows, B):
    dims = CacheDims(fmt, heads, k_dim, v_dim, 1, 0, 1.0, 1.0)
    return _lib.lib().mxfp4_cache_attend_workspace_bytes(ctypes.byref(dims), q_heads, rows, B)


def _vectors(t, name, heads, dim):
    """(address, elements from row to row, from head to head; the stride of a dimension of one entry says nothing)."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim or t.stride(2) != 1 and dim > 1:
        raise ValueError(f"{name}: [rows, {heads}, {dim}], last dimension contiguous")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else heads * dim, t.stride(1) if heads > 1 else dim


def _check_table(page_table):
    """(row stride, rows, columns)."""
    if page_table.dtype != torch.int32 or page_table.dim() != 2:
        raise ValueError("page_table: int32 [B, pages]")
    B, P = page_table.shape
    _need_int32(B, P)
    if P > 1 and page_table.stride(1) != 1 or B > 1 and page_table.stride(0) < P:
        raise ValueError("page_table's last dimension must be contiguous, its rows must not overlap")
    return page_table.stride(0) if B > 1 else P, B, P


def _check_list(t, name, n):
    _need(t.dtype == torch.int32 and t.shape == (n,) and t.is_contiguous(), f"{name}: contiguous int32 [{n}]")


class PagedCache:
    """A paged cache of keys and values (or one plane, v_dim=0) held in a block format.

    A token has `heads` vectors of k_dim (and v_dim; None: k_dim) elements; page_size tokens make a page.
    The memory is four uint8 tensors k_q, k_s, v_q, v_s (codes [num_pages, page_size, heads, dim/2], MXFP8: dim;
    scales [num_pages, page_size, heads, dim/32], NVFP4: dim/16), allocated as zeros or given as `storage`.  They and
    `dims` (a copy of the sizes) cannot be rebound; another memory is another PagedCache."""

    def __init__(self, num_pages, page_size, heads, k_dim, v_dim=None, fmt=FMT_MXFP8, k_global_scale=1.0,
                 v_global_scale=1.0, storage=None, device=None):
        v_dim = k_dim if v_dim is None else v_dim
        _need_int32(fmt, heads, k_dim, v_dim, page_size)
        self._dims = CacheDims(fmt, heads, k_dim, v_dim, page_size, num_pages, k_global_scale, v_global_scale)
        sizes = (ctypes.c_size_t * 4)()
        check("mxfp4_cache_bytes", _lib.lib().mxfp4_cache_bytes(ctypes.byref(self._dims), sizes))
        per = 1 if fmt == FMT_MXFP8 else 2
        shapes = [(num_pages, page_size, heads, d // by) for d in (k_dim, v_dim) for by in (per, _GROUP[fmt])]
        if storage is None:
            device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
            storage = [torch.zeros(s, dtype=torch.uint8, device=device) if s[-1] else None for s in shapes]
        _need(len(storage) == 4, "storage: (k_q, k_s, v_q, v_s)")
        for n, t, s in zip(("k_q", "k_s", "v_q", "v_s"), storage, shapes):
            if s[-1] == 0:
                _need(t is None, f"{n} must be None when v_dim is 0")
                continue
            _need(t is not None and t.dtype == torch.uint8 and t.shape == s and t.is_contiguous(),
                  f"{n}: contiguous uint8 {list(s)}")
        self._storage = k_q, *_ = tuple(storage)
        self._gpu = _gpu_of("k_q", *storage)
        self._device = k_q.device
        self._heads, self._k_dim, self._v_dim = heads, k_dim, v_dim
        self._dref = ctypes.byref(self._dims)

    # what the kernels' bounds were checked against: read only
    dims = property(lambda self: CacheDims.from_buffer_copy(self._dims))
    k_q = property(lambda self: self._storage[0])
    k_s = property(lambda self: self._storage[1])
    v_q = property(lambda self: self._storage[2])
    v_s = property(lambda self: self._storage[3])

    def _memory(self):
        """The tensors' addresses now: their memory may have moved since the last call."""
        k_q, k_s, v_q, v_s = self._storage
        if v_q is None:
            return k_q.data_ptr(), k_s.data_ptr(), None, None
        return k_q.data_ptr(), k_s.data_ptr(), v_q.data_ptr(), v_s.data_ptr()

    def _index(self, page_table, cu_rows, start):
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or cu_rows.dtype != torch.int32:
            raise ValueError("page_table: int32 [B, pages], cu_rows: int32 [B + 1]")
        B, P = page_table.shape
        if (B | P) >> 31:
            _need_int32(B, P)
        if P > 1 and page_table.stride(1) != 1 or B > 1 and page_table.stride(0) < P:
            raise ValueError("page_table's last dimension must be contiguous, its rows must not overlap")
        if cu_rows.shape != (B + 1,) or not cu_rows.is_contiguous():
            raise ValueError("cu_rows: contiguous int32 [B + 1]")
        if start is not None and (start.dtype != torch.int32 or start.shape != (B,) or not start.is_contiguous()):
            raise ValueError("start: contiguous int32 [B]")
        return cu_rows.data_ptr(), _ptr(start), page_table.data_ptr(), page_table.stride(0) if B > 1 else P, B, P

    def _rows(self, t, name, dim):
        heads = self._heads
        if t.dtype != torch.bfloat16 or t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim or t.stride(2) != 1:
            raise ValueError(f"{name}: bf16 [rows, {heads}, {dim}], last dimension contiguous")
        # the stride of a dimension of one entry says nothing
        return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else heads * dim, t.stride(1) if heads > 1 else dim

    def _planes(self, k, v):
        if (v is None) != (self._v_dim == 0):
            raise ValueError("v goes with v_dim > 0, and only with it")
        k_args = self._rows(k, "k", self._k_dim)
        if v is None:
            return *k_args, None, 0, 0
        _need(v.shape[0] == k.shape[0], "k and v must have the same number of rows")
        return *k_args, *self._rows(v, "v", self._v_dim)

    def write(self, k, v, page_table, cu_rows, start=None):
        """Quantizes the rows of k [rows, heads, k_dim] and v (None with v_dim=0) into the cache.  Rows
        [cu_rows[b], cu_rows[b+1]) are sequence b's positions start[b], start[b]+1, ... (start None: from 0);
        position i lives in page page_table[b, i // page_size].  Rows outside every sequence, and positions without
        a page (past the table, or a page number outside the cache), are passed over.  Two rows of one call must not
        share a slot.  Rows and heads may be strided, by multiples of 8 elements, and start on 16 bytes."""
        _gpu_of("the cache", self._storage[0], k, v, page_table, cu_rows, start)
        index = self._index(page_table, cu_rows, start)
        planes = self._planes(k, v)
        _call(self._gpu, "mxfp4_cache_write", self._dref, *planes, k.shape[0], *index, *self._memory())

    def read(self, page_table, cu_rows, start=None, rows=None, k_out=None, v_out=None):
        """Reads rows back as bf16: (k [rows, heads, k_dim], v or None), rows and positions as in `write`.  Give
        `rows` (the outputs are allocated; rows outside every sequence are then undefined) or the outputs, whose
        rows outside every sequence are left as they were and whose vectors must not overlap.
        Positions without a page read as zeros."""
        index = self._index(page_table, cu_rows, start)
        given = k_out is not None
        if not given:
            _need(rows is not None and rows >= 0 and v_out is None, "give rows, or the outputs")
            k_out = torch.empty((rows, self._heads, self._k_dim), dtype=torch.bfloat16, device=self._device)
            if self._v_dim:
                v_out = torch.empty((rows, self._heads, self._v_dim), dtype=torch.bfloat16, device=self._device)
        else:
            _check_given(k_out, v_out)
        _gpu_of("the cache", self._storage[0], k_out, v_out, page_table, cu_rows, start)
        planes = self._planes(k_out, v_out)
        _need(rows is None or rows == k_out.shape[0], "rows must be the outputs' rows")
        _call(self._gpu, "mxfp4_cache_read", self._dref, *self._memory(), k_out.shape[0], *index, *planes)
        if given:
            _changed((k_out,) if v_out is None else (k_out, v_out))
        return k_out, v_out

    def attend(self, q, page_table, cu_rows, start=None, tree_mask=None, scale=None, out=None, out_dtype=torch.bfloat16):
        """Attention of rows whose keys and values `write` has put into the cache, with the same cu_rows, start and
        page_table: one new token a sequence, a chunk of a prompt, or a tree of drafted tokens.

        q bf16 [rows, q_heads, k_dim] (q_heads a multiple of heads; rows and heads may be strided, by multiples of 8
        elements, and start on 16 bytes).  A row sees the positions below its sequence's start, and of the sequence's own
        rows those up to itself, or with tree_mask (bool or uint8 [rows, W], rows may be strided) those j < W with
        tree_mask[row, j] set: j counts from the sequence's first row.  Positions without a page are not seen.  scale
        (None: k_dim ** -0.5) multiplies the scores.  Returns [rows, q_heads, v_dim] in out_dtype (bfloat16 or float32);
        bfloat16: the softmax's weights are rounded to it before they meet the values where a sequence has more than 16 rows
        a key head on average; float32, or fewer rows: 2^-16 of them are lost;
        a row that sees nothing gets zeros, NaN in a query or in what it sees gives NaN.  Rows outside every sequence are
        undefined, or in `out` (strided like q) left as they were; `out` and q must not overlap.  Forward only: a q that
        asks for a gradient is refused."""
        _gpu_of("the cache", self._storage[0], q, page_table, cu_rows, start, tree_mask, out)
        if torch.is_grad_enabled() and q.requires_grad:
            raise ValueError("attend has no backward pass: detach q, or call it under torch.no_grad()")
        _no_tangent("attend", q)
        index = self._index(page_table, cu_rows, start)
        _need(self._v_dim > 0, "attend needs a cache with keys and values (v_dim > 0)")
        _need(q.dtype == torch.bfloat16 and q.dim() == 3, f"q: bf16 [rows, q_heads, {self._k_dim}]")
        rows, q_heads = q.shape[:2]
        _need_int32(q_heads)
        _need(q_heads > 0 and q_heads % self._heads == 0, "q_heads must be a multiple of the cache's heads")
        q_args = _vectors(q, "q", q_heads, self._k_dim)
        given = out is not None
        if not given:
            out_fp32 = _check_out(out_dtype)
            out = torch.empty((rows, q_heads, self._v_dim), dtype=out_dtype, device=self._device)
        else:
            out_fp32 = _check_out(out.dtype)
            _need(out.shape[0] == rows, "out must have q's rows")
            _check_given(out)
        mask, ld_mask, W = None, 0, 0
        if tree_mask is not None:
            _need(tree_mask.dtype in (torch.bool, torch.uint8) and tree_mask.dim() == 2 and tree_mask.shape[0] == rows,
                  "tree_mask: bool or uint8 [rows, W]")
            W = tree_mask.shape[1]
            _need_int32(W)
            _need(W <= 1 or tree_mask.stride(1) == 1, "tree_mask's last dimension must be contiguous")
            ld_mask = tree_mask.stride(0) if rows > 1 else W
            _need(ld_mask >= W, "tree_mask's rows must not overlap")
            # a mask without columns hides all drafts: it must not become the absent mask
            mask = tree_mask.data_ptr() or q.data_ptr()
        scale = self._k_dim ** -0.5 if scale is None else scale
        nws = _attend_workspace(self._dims.fmt, self._heads, self._k_dim, self._v_dim, q_heads, rows, index[4])
        if nws == 0:
            raise ValueError("invalid attention arguments (k_dim and v_dim are at most 256)")
        ws = torch.empty(nws, dtype=torch.uint8, device=self._device)
        _call(self._gpu, "mxfp4_cache_attend", self._dref, *self._memory(), *q_args, q_heads, rows, *index, mask, ld_mask, W,
              scale, *_vectors(out, "out", q_heads, self._v_dim), out_fp32, ws.data_ptr(), nws)
        if given:
            _changed(out)
        return out

    def compact(self, page_table, start, path):
        """Moves the accepted drafts of each sequence together: position start[b] + i takes what position
        start[b] + path[b, i] held.  path int32 [B, W] (rows may be strided): indices of accepted drafts in increasing
        order, ended by a negative entry, by one that does not increase, or by the last column; start int32 [B] as in
        `write`.  Returns the new lengths int32 [B], start + the number of accepted drafts.  Positions without a page are
        passed over.  Sequences must not share the pages that drafts lie in (`PagePool` gives each its own)."""
        gpu = _gpu_of("the cache", self._storage[0], page_table, start, path)
        ld, B, P = _check_table(page_table)
        _check_list(start, "start", B)
        _need(path.dtype == torch.int32 and path.dim() == 2 and path.shape[0] == B, "path: int32 [B, W]")
        W = path.shape[1]
        _need_int32(W)
        _need(W <= 1 or path.stride(1) == 1, "path's last dimension must be contiguous")
        ld_path = path.stride(0) if B > 1 else W
        _need(ld_path >= W, "path's rows must not overlap")
        lengths = torch.empty(B, dtype=torch.int32, device=self._device)
        _call(gpu, "mxfp4_cache_compact", self._dref, start.data_ptr(), path.data_ptr(), ld_path, W, page_table.data_ptr(),
              ld, B, P, lengths.data_ptr(), *self._memory())
        return lengths

    def copy_pages(self, src, dst, rows=None):
        """Copies the first rows[i] tokens (None: all) of page src[i] to page dst[i]; all int32 [n].  A pair with a page
        outside the cache is passed over.  A destination must not be in the lists a second time."""
        gpu = _gpu_of("the cache", self._storage[0], src, dst, rows)
        n = src.shape[0] if src.dim() == 1 else -1
        _need_int32(n)
        for t, name in ((src, "src"), (dst, "dst"), (rows, "rows")):
            if t is not None:
                _check_list(t, name, n)
        _call(gpu, "mxfp4_cache_copy_pages", self._dref, src.data_ptr(), dst.data_ptr(), _ptr(rows), n, *self._memory())


# ------------------------------------------------------------------------------------------------
# Page pool.


@functools.lru_cache(maxsize=256)
def _pool_workspace(num_pages, n, columns):
    return _lib.lib().mxfp4_pool_workspace_bytes(num_pages, n, columns)


class PagePool:
    """Which pages of one or more caches are in use (a model's layers share page tables, and so a pool), on the device.

    refs int32 [num_pages]: how many rows of the page tables hold each page, 0: free; zeros, or given where pages are
    held already.  A row of a page table holds its leading entries in [0, num_pages); the others are -1.  Free pages are
    handed out in increasing order, to rows in increasing order.  Tables and refs are changed in place, and all caches'
    pages that have to be copied are.  Calls on one pool must be ordered (one stream)."""

    def __init__(self, *caches, refs=None):
        _need(len(caches) > 0 and all(isinstance(c, PagedCache) for c in caches), "give the caches whose pages are pooled")
        d = caches[0].dims
        for c in caches[1:]:
            other = c.dims
            _need((other.num_pages, other.page_size) == (d.num_pages, d.page_size),
                  "the caches must have the same number of pages and page size")
        self._caches, self._pages, self._page_size = caches, d.num_pages, d.page_size
        device = caches[0].k_q.device
        if refs is None:
            refs = torch.zeros(d.num_pages, dtype=torch.int32, device=device)
        _check_list(refs, "refs", d.num_pages)
        self._refs = refs
        self._gpu = _gpu_of("the cache", *(c.k_q for c in caches), refs)
        self._device = device

    # what the kernels' bounds were checked against: read only
    refs = property(lambda self: self._refs)
    caches = property(lambda self: self._caches)

    def _change(self, fn, page_table, n, lists):
        ld, B, P = _check_table(page_table)
        nws = _pool_workspace(self._pages, n, P)
        if nws == 0:
            raise ValueError("invalid page pool arguments")
        # the workspace and copies [3, n] behind it (a whole number of 256 bytes)
        ws = torch.empty(nws + 12 * n, dtype=torch.uint8, device=self._device)
        missing = torch.empty((), dtype=torch.int32, device=self._device)
        copies = ws.data_ptr() + nws
        _call(self._gpu, fn, self._pages, self._page_size, self._refs.data_ptr(), page_table.data_ptr(), ld, B, P, *lists,
              copies, missing.data_ptr(), copies - nws, nws)
        for c in self._caches:
            _call(self._gpu, "mxfp4_cache_copy_pages", c._dref, copies, copies + 4 * n, copies + 8 * n, n, *c._memory())
        return missing

    def resize(self, page_table, lengths):
        """Row b of page_table (int32 [B, pages]) then holds the pages of lengths[b] tokens (int32 [B]; negative: the row
        is left alone; as many pages as the table has columns at most): pages are taken, or given back (0: all).  Where
        the length ends inside a page that the row shares, it gets a copy of its own.  Returns int32, 0-dim: the pages that
        were wanted when none was free; their entries are -1, where `write` and `attend` pass over them.  That holds for a
        shared page that was to be replaced too: the row gives up its tokens there, unless no other row holds the page
        any more, whose last row then keeps it.  (Make room first where a row must not lose them.)"""
        _gpu_of("the cache", self._refs, page_table, lengths)
        n = page_table.shape[0] if page_table.dim() == 2 else 0
        _check_list(lengths, "lengths", n)
        return self._change("mxfp4_pool_resize", page_table, n, (lengths.data_ptr(),))

    def fork(self, page_table, src, dst, lengths):
        """Row dst[i] of page_table gives its pages back and continues from the first lengths[i] tokens of row src[i]
        (all int32 [n]): whole pages are shared, the last one is copied where they end inside it.  A pair is passed over
        when a row is outside the table, the length is negative, dst[i] is a source too, or an earlier pair has it.
        Returns as `resize`."""
        _gpu_of("the cache", self._refs, page_table, src, dst, lengths)
        n = src.shape[0] if src.dim() == 1 else -1
        _need_int32(n)
        for t, name in ((src, "src"), (dst, "dst"), (lengths, "lengths")):
            _check_list(t, name, n)
        return self._change("mxfp4_pool_fork", page_table, n, (src.data_ptr(), dst.data_ptr(), lengths.data_ptr(), n))
