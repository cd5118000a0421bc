"""float64 references of the router's losses and of its dense backward, written
from the definitions in include/mok.h (test infrastructure; no code shared with
the HIP path)."""
from __future__ import annotations

import numpy as np


def softmax(logits):
    """(p, lse) row by row; a row of nothing but -inf has zeros for both."""
    top = logits.max(1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    ex = np.exp(logits - top)
    den = ex.sum(1, keepdims=True)
    none = den == 0
    safe = np.where(none, 1.0, den)
    return ex / safe, np.where(none, 0.0, top + np.log(safe))[:, 0]


def losses(logits, ids, mask=None):
    """dict of losses [2], counts [E], prob_sum [E], n (and p, lse, m of the tokens)."""
    T, E = logits.shape
    m = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    p, lse = softmax(np.where(m[:, None], logits, 0.0))
    counts = np.zeros(E, np.int64)
    for row in ids[m]:
        for e in row:
            if 0 <= e < E:
                counts[e] += 1
    n, k = int(m.sum()), ids.shape[1]
    prob = p[m].sum(0)
    out = np.zeros(2)
    if n:
        out[:] = E / (k * n * n) * (counts * prob).sum(), (lse[m] ** 2).sum() / n
    return {"losses": out, "counts": counts, "prob_sum": prob, "n": n, "p": p, "lse": lse, "m": m}


def losses_backward(r, ids, d_losses, w=None, g=None):
    """d_logits [T][E] from r = losses(...)."""
    p, m, n, k = r["p"], r["m"], r["n"], ids.shape[1]
    T, E = p.shape
    d = np.zeros((T, E))
    if n:
        c = r["counts"].astype(np.float64)
        d = d_losses[0] * E / (k * n * n) * p * (c - (p * c).sum(1, keepdims=True)) + d_losses[1] * 2 / n * p * r["lse"][:, None]
        d = np.where(m[:, None], d, 0.0)
    if w is not None:
        sel = w * (g - (w * g).sum(1, keepdims=True))
        for t in range(T):
            for j in range(k):
                if 0 <= ids[t, j] < E:
                    d[t, ids[t, j]] += sel[t, j]
    return d


def logits_backward(x, wr, dl, residual=None):
    dx = dl @ wr
    return (dx if residual is None else dx + residual), dl.T @ x
