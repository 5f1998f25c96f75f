"""Oracle: attention over the paged cache in a block format, in float64.

Test infrastructure only (see the package docstring).  Keys and values are the cache's (code * scale / global scale, not
rounded to bf16); row t of sequence b is its draft i and sees the positions below start[b], and of the drafts those that
the mask marks or, without one, those up to itself [DEF].
"""

import numpy as np


def seen_ref(i, n, start, mask_row, table_row, page_size, num_pages):
    """(position, slot) of what draft i of a sequence of n drafts sees, position by position."""
    out = []
    for pos in range(0, start + n):
        j = pos - start
        if j >= 0 and (j > i if mask_row is None else j >= len(mask_row) or not mask_row[j]):
            continue
        p = pos // page_size
        page = int(table_row[p]) if p < len(table_row) else -1
        if 0 <= page < num_pages:
            out.append((pos, page * page_size + pos % page_size))
    return out


def attend_ref(q, k, v, cu, start, table, page_size, mask=None, scale=None):
    """q float64 [rows, Hq, dk]; k, v float64 [slots, H, d] (decoded); cu, start per sequence; mask [rows, W] or None.
    Returns (out, weight, score), float64: weight = sum_j p_j |v_j|, what an error of the weights is multiplied by;
    score [rows, Hq] = the largest sum_i |q_i k_ji| * |scale|, what an error of the products is relative to.  Rows outside
    every sequence are NaN."""
    rows, hq, dk = q.shape
    heads, num_pages = k.shape[1], k.shape[0] // page_size
    scale = dk ** -0.5 if scale is None else scale
    out = np.full((rows, hq, v.shape[2]), np.nan)
    weight, score = np.zeros_like(out), np.zeros((rows, hq))
    for b in range(len(cu) - 1):
        for t in range(max(0, int(cu[b])), min(rows, int(cu[b + 1]))):
            n, i = int(cu[b + 1]) - int(cu[b]), t - int(cu[b])
            at = [s for _, s in seen_ref(i, n, 0 if start is None else int(start[b]), None if mask is None else mask[t], table[b],
                                         page_size, num_pages)]
            out[t] = 0.0
            if not at:
                continue
            for h in range(hq):
                g = h // (hq // heads)
                s = k[at, g] @ q[t, h] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[t, h] = p @ v[at, g]
                weight[t, h] = p @ np.abs(v[at, g])
                score[t, h] = np.max(np.abs(k[at, g]) @ np.abs(q[t, h])) * abs(scale)
    return out, weight, score
