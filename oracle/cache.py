"""Oracle: the paged cache in a block format.

Test infrastructure only (see the package docstring).  Rows are quantized with the quantizers' rules (MXFP4 and
NVFP4 as the matrix quantizers, MXFP8 as the quantized activations) and placed through a page table [DEF].
"""

import numpy as np

from . import quant as Q


def slots_ref(rows, cu, start, table, page_size, num_pages):
    """Row by row, in plain Python: the slot of each row, -1 where its position has no page, None where the row
    belongs to no sequence."""
    out = [None] * rows
    for b in range(len(cu) - 1):
        for t in range(max(0, int(cu[b])), min(rows, int(cu[b + 1]))):
            pos = t - int(cu[b]) + (0 if start is None else int(start[b]))
            page = int(table[b][pos // page_size]) if 0 <= pos < len(table[b]) * page_size else -1
            out[t] = page * page_size + pos % page_size if 0 <= page < num_pages else -1
    return out


def encode_ref(x_bits, fmt, gs):
    """x_bits uint16 [..., D] -> (codes, scales) as the cache holds them."""
    D = x_bits.shape[-1]
    flat = np.ascontiguousarray(x_bits).reshape(-1, D)
    if fmt == "mxfp4":
        q, s = Q.quantize_ref(flat)
    elif fmt == "nvfp4":
        q, s = Q.nvfp4_quantize_ref(flat, gs)
    else:
        q, s = Q.mxfp8_quantize_values_ref(Q.bf16_to_f64(flat).astype(np.float32))
    return q.reshape(*x_bits.shape[:-1], -1), s.reshape(*x_bits.shape[:-1], -1)


def decode_ref(q, s, fmt, gs):
    """The cached values in float64: code * scale (NVFP4: / global scale, a binary32 number; the quotient's rounding to
    float64 is the only one).  A value that is read back is one of these, rounded to bf16."""
    if fmt == "mxfp4":
        return Q.dequant_ref(q, s)
    if fmt == "mxfp8":
        return Q.mxfp8_dequant_ref(q, s)
    codes = Q.unpack_codes(q)
    v = np.where(codes & 8, -1.0, 1.0) * Q.E2M1_MAGNITUDES[codes & 7]
    return v * np.repeat(Q.E4M3_MAGNITUDES[s].astype(np.float64), Q.NV_BLOCK, axis=-1) / float(np.float32(gs))


def bf16_bits(v):
    """Numbers (not NaN) -> bf16 bits in one rounding, nearest even; infinities stay."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    step = np.ldexp(1.0, np.maximum(np.frexp(np.where(np.isfinite(a), a, 0.0))[1] - 1, -126) - 7)
    r = np.where(np.isfinite(a), np.rint(a / step) * step, a)
    r = np.copysign(np.where(r >= 2.0 ** 128, np.inf, r), v).astype(np.float32)  # exact: eight bits
    return (r.view(np.uint32) >> np.uint32(16)).astype(np.uint16)
