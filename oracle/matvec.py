"""Oracle: products with 4-bit weights in the standard layout, dense and per routed pair, in float64.

Test infrastructure only (see the package docstring).

    y = x W^T / global_scale + b,   W = dequantized MXFP4 (global_scale 1) or NVFP4 codes and scales

[DEF: the linear layer with 4-bit weights and 16-bit activations (W4A16), and the experts' products of the MoE
layer: rows [w1; w3], SwiGLU = silu(w1 half) * (w3 half)]
"""

import numpy as np

from .quant import bf16_to_f64, dequant_ref, nvfp4_dequant_ref


def weights_ref(w_q, w_s, global_scale=None):
    """Weights as float64; NVFP4 where a global scale is given."""
    return dequant_ref(w_q, w_s) if global_scale is None else nvfp4_dequant_ref(w_q, w_s, global_scale)


def matvec_ref(x_bits, w_q, w_s, b=None, global_scale=None):
    """x_bits uint16 [M, K] bf16, b float64 [N] or None.  Returns (y [M, N], sum_k |x W| [M, N])."""
    x, w = bf16_to_f64(x_bits), weights_ref(w_q, w_s, global_scale)
    y = x @ w.T
    return (y if b is None else y + b[None, :]), np.abs(x) @ np.abs(w).T


def expert_matvec_ref(x_bits, w_q, w_s, ids, shared_rows, b=None, global_scales=None):
    """ids int [T, k]; pair p = t * k + j multiplies row t (shared_rows) or row p of x.  Returns (y [T * k, N],
    sum_k |x W|)."""
    ids = np.asarray(ids)
    k = ids.shape[1]
    y, mag = [], []
    for p, e in enumerate(ids.reshape(-1)):
        r = p // k if shared_rows else p
        a, m = matvec_ref(x_bits[r:r + 1], w_q[e], w_s[e], None if b is None else b[e],
                          None if global_scales is None else global_scales[e])
        y.append(a[0])
        mag.append(m[0])
    return np.array(y), np.array(mag)


def swiglu_ref(h):
    """silu(first half of the columns) * second half."""
    g, u = np.split(h, 2, axis=-1)
    return g / (1.0 + np.exp(-g)) * u
