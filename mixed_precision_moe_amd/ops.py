"""The balance loss, the 4-bit matrix-vector products and the block-quantized paged cache: the torch binding of
their C entry points.  Like the rest of the binding it checks dtypes, shapes and devices, allocates
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
    if y is None:
        out_fp32 = _check_out(out_dtype)
        y = torch.empty((P, width), dtype=out_dtype, device=x.device)
    else:
        out_fp32 = _check_out(y.dtype)
        _need(y.shape == (P, width) and y.is_contiguous(), "y: contiguous [P, N] (swiglu: [P, N/2])")
    _call(gpu, "fp4_expert_matvec", fmt, w_q.data_ptr(), w_s.data_ptr(), _ptr(global_scales), E, N, K, _ptr(bias),
          is_fp32, x.data_ptr(), ldx, top_k, expert_offsets.data_ptr(), sorted_pairs.data_ptr(), P, 1 if swiglu else 0,
          y.data_ptr(), out_fp32)
    return y


# ------------------------------------------------------------------------------------------------
# Paged cache.


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
        if k_out is None:
            _need(rows is not None and rows >= 0 and v_out is None, "give rows, or the outputs")
            k_out = torch.empty((rows, self._heads, self._k_dim), dtype=torch.bfloat16, device=self._device)
            if self._v_dim:
                v_out = torch.empty((rows, self._heads, self._v_dim), dtype=torch.bfloat16, device=self._device)
        _gpu_of("the cache", self._storage[0], k_out, v_out, page_table, cu_rows, start)
        planes = self._planes(k_out, v_out)
        _need(rows is None or rows == k_out.shape[0], "rows must be the outputs' rows")
        _call(self._gpu, "mxfp4_cache_read", self._dref, *self._memory(), k_out.shape[0], *index, *planes)
        return k_out, v_out
