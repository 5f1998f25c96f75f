"""Oracle: the router's balance loss, its per-expert counts and its gradient, in float64.

Test infrastructure only (see the package docstring).  The pages never write the loss down; this library adopts
the usual definition [DEF]: with p_t the softmax of token t's logits, n_e the number of pairs of expert e and V the
number of tokens that count,

    loss = E / (k V^2) * sum_e n_e * sum_t p_te,

the counts being constants of the gradient.
"""

import numpy as np


def softmax_rows(logits):
    """Row softmax in float64; a row of -inf throughout gives zeros (nothing to share out)."""
    l = np.asarray(logits, dtype=np.float64)
    top = l.max(axis=1, keepdims=True)
    p = np.exp(l - np.where(np.isfinite(top), top, 0.0))
    s = p.sum(axis=1, keepdims=True)
    return np.where(s > 0, p / np.where(s > 0, s, 1.0), 0.0)


def balance_ref(logits, ids, mask=None, g=1.0):
    """logits [T, E], ids int [T, k] (outside [0, E): dropped), mask bool [T] or None.
    Returns (loss, counts int64 [E], gradient float64 [T, E] of g * loss)."""
    logits = np.asarray(logits)
    ids = np.asarray(ids)
    T, E = logits.shape
    keep = np.arange(T) if mask is None else np.flatnonzero(np.asarray(mask))
    flat = ids[keep].reshape(-1)
    counts = np.bincount(flat[(flat >= 0) & (flat < E)].astype(np.int64), minlength=E)
    grad = np.zeros((T, E))
    V, k = keep.size, ids.shape[1]
    if V == 0:
        return 0.0, counts, grad
    p = softmax_rows(logits[keep])
    c = E / (k * float(V) ** 2)
    loss = c * float((counts * p.sum(axis=0)).sum())
    # a constant added to every n_e drops out of the bracket where sum_e p_te = 1; the mean is taken off, which
    # also says what a row without probabilities gets (0)
    d = c * (counts - counts.mean())
    grad[keep] = g * p * (d - (p * d).sum(axis=1, keepdims=True))
    return loss, counts, grad
