"""Rotary positions: the torch binding of mxfp4_rotary, and the frequencies of a layer's configuration."""

import math

import torch

from .ops import _call, _changed, _gpu_of, _need, _need_int32, _no_tangent, _vectors


def rotary_frequencies(dim, base=10000.0, scaling=None):
    """(angle per position of each of the dim / 2 pairs, float64 on the host; factor of the turned vectors).

    base ** (-2 i / dim), changed by `scaling` for contexts that are longer than a model was trained on:
      None                      as they are
      kind="linear", factor     divided by factor
      kind="base", factor       base * factor ** (dim / (dim - 2)): the slowest is divided by factor, the fastest kept
      kind="ramp", factor, length, fast=32, slow=1, magnitude=1 + 0.1 ln(factor) (1 for factors below 1)
          pairs that turn more than `fast` times over `length` positions are kept, those that turn fewer than `slow`
          times divided by factor, with a ramp over the pairs between; queries and keys are multiplied by magnitude
      kind="bands", factor, length, low=1, high=4
          the same between length / high and length / low positions a turn, with a ramp over the turns themselves"""
    _need(isinstance(dim, int) and dim >= 2 and dim % 2 == 0, "dim must be even")
    _need(base > 0, "base must be positive")
    s = dict(scaling or {})
    kind, factor = s.pop("kind", None), s.pop("factor", 1.0)
    _need(factor > 0, "factor must be positive")
    if kind == "base":
        _need(dim > 2, "kind='base' needs more than one pair")
        base = base * factor ** (dim / (dim - 2))
    f = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    magnitude = 1.0
    if kind == "linear":
        f = f / factor
    elif kind == "ramp":
        _need("length" in s, "kind='ramp' needs length")
        _need(base != 1, "kind='ramp' needs a base other than 1")
        length, fast, slow = s.pop("length"), s.pop("fast", 32.0), s.pop("slow", 1.0)
        magnitude = s.pop("magnitude", 1.0 + 0.1 * math.log(max(factor, 1.0)))
        # the index of a pair that turns n times over the length
        pair = lambda n: dim * math.log(length / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
        low, high = max(0, math.floor(pair(fast))), min(dim - 1, math.ceil(pair(slow)))
        ramp = ((torch.arange(dim // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
    elif kind == "bands":
        _need("length" in s, "kind='bands' needs length")
        length, low, high = s.pop("length"), s.pop("low", 1.0), s.pop("high", 4.0)
        _need(high > low, "high must be above low")
        kept = ((length * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * kept + f / factor * (1 - kept)
    else:
        _need(kind in (None, "base"), f"unknown scaling {kind!r}")
    _need(not s, f"unknown scaling options {sorted(s)}")
    return f, magnitude


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, handle, inverse, positions, *tensors):
        ctx.handle, ctx.inverse = handle, inverse
        ctx.save_for_backward(positions)
        ctx.set_materialize_grads(False)
        made = handle._apply(tensors, positions, inverse)
        ctx.mark_non_differentiable(*(x for x, asks in zip(made, ctx.needs_input_grad[3:]) if not asks))
        return made

    @staticmethod
    def backward(ctx, *grads):
        # a rotation's gradient is the rotation back (by the same magnitude), itself differentiable
        positions, = ctx.saved_tensors
        given = [g if g.dim() == 3 and g.stride(2) == 1 else g.contiguous() for g in grads if g is not None]
        back = iter(ctx.handle._turn(given, positions, not ctx.inverse) if given else ())
        return (None, None, None, *(None if g is None else next(back) for g in grads))


class Rotary:
    """Rotary positions of a layer: its frequencies, on the device.

    Elements [offset, offset + dim) of each head's vector are turned, pair i by positions * frequency i: elements
    (i, i + dim / 2), or (2i, 2i + 1) with interleaved.  base and scaling as in `rotary_frequencies`, or freqs: the
    frequencies themselves (float64 [dim / 2], with `magnitude`)."""

    def __init__(self, dim, base=10000.0, *, interleaved=False, offset=0, scaling=None, freqs=None, magnitude=None,
                 device=None):
        if freqs is None:
            freqs, own = rotary_frequencies(dim, base, scaling)
            magnitude = own if magnitude is None else magnitude
        else:
            _need(scaling is None, "scaling changes frequencies that are made here: give it, or freqs")
            freqs = torch.as_tensor(freqs, dtype=torch.float64)
            _need(dim % 2 == 0 and freqs.shape == (dim // 2,), "freqs: one for each pair")
        _need(2 <= dim <= 2048 and offset >= 0, "2 <= dim <= 2048, offset >= 0")
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self._turns = (freqs / (2 * math.pi)).to(device).contiguous()
        self._dim, self._offset, self._interleaved = dim, offset, 1 if interleaved else 0
        self._magnitude = 1.0 if magnitude is None else float(magnitude)
        _need(math.isfinite(self._magnitude), "magnitude must be finite")

    def _apply(self, tensors, positions, inverse, out=None):
        q, k = tensors if len(tensors) == 2 else (tensors[0], None)
        gpu = _gpu_of("q", q, positions, self._turns, k)
        dtype = q.dtype
        _need(dtype == torch.bfloat16 or dtype == torch.float32, "q and k: bf16 or fp32")
        _need(q.dim() == 3 and (k is None or k.dim() == 3), "q and k: [rows, heads, head_dim]")
        rows, heads, dim = q.shape
        if (dim | heads) >> 31:
            _need_int32(dim, heads)
        _need(heads > 0, "q must have a head")
        _need(self._offset + self._dim <= dim, "the turned part must lie inside head_dim")
        _need(positions.dtype == torch.int32 and positions.shape == (rows,) and positions.is_contiguous(),
              "positions: contiguous int32 [rows]")
        q_args, k_args, k_heads = _vectors(q, "q", heads, dim), (None, 0, 0), 0
        if k is not None:
            k_heads = k.shape[1]
            _need_int32(k_heads)
            _need(k.dtype == dtype and k.shape[0] == rows, "q and k must have the same rows and dtype")
            _need(k_heads > 0, "k must have a head")
            k_args = _vectors(k, "k", k_heads, dim)
        if out is None:
            q_out = torch.empty((rows, heads, dim), dtype=dtype, device=q.device)
            made, q_to, k_to = (q_out,), (q_out.data_ptr(), heads * dim, dim), (None, 0, 0)
            if k is not None:
                k_out = torch.empty((rows, k_heads, dim), dtype=dtype, device=q.device)
                made, k_to = (q_out, k_out), (k_out.data_ptr(), k_heads * dim, dim)
        else:
            made, q_to, k_to = out, q_args, k_args
        _call(gpu, "mxfp4_rotary", self._turns.data_ptr(), positions.data_ptr(), rows, dim, self._dim, self._offset,
              self._interleaved, self._magnitude, 1 if inverse else 0, 1 if dtype == torch.float32 else 0, *q_args, heads,
              *q_to, *k_args, k_heads, *k_to)
        return made

    def _turn(self, tensors, positions, inverse):
        _no_tangent("Rotary", *tensors)
        if torch.is_grad_enabled() and (tensors[0].requires_grad or tensors[-1].requires_grad):
            return _Rotary.apply(self, inverse, positions, *tensors)
        return self._apply(tensors, positions, inverse)

    def __call__(self, q, k, positions, inplace=False):
        """q [rows, q_heads, head_dim] and k [rows, k_heads, head_dim] (or None), bf16 or fp32, rows and heads strided as
        they like; positions int32 [rows].  Returns both turned (contiguous), differentiable in q and k any number of
        times (backward; forward-mode tangents are refused); with inplace, in their own memory (not where a gradient is
        asked for, and a backward pass that saved them is then refused by autograd; they must not overlap; the elements
        outside the turned part are not touched).  To capture the backward pass into a graph, drop every eager autograd
        graph of the same leaves first, as torch asks for any backward pass."""
        tensors = (q,) if k is None else (q, k)
        if inplace:
            _no_tangent("Rotary", *tensors)
            _need(not (torch.is_grad_enabled() and any(t.requires_grad for t in tensors)),
                  "inplace has no backward pass: a gradient needs the form that is not in place")
            _need(k is None or q.shape[0] == 0 or q.data_ptr() != k.data_ptr(), "in place, q and k must not overlap")
            out = self._apply(tensors, positions, False, out=tensors)
            _changed(tensors)
        else:
            out = self._turn(tensors, positions, False)
        return out[0], None if k is None else out[1]
