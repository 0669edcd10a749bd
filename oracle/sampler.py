"""Oracle of the sampler (test infrastructure only; see the package docstring).

One row at a time in float64: sort by falling logit (equal logits by rising
index), weigh, cut by top-k, top-p and min-p in turn, and walk the cumulative
weights to u times their sum.  `margin` is how far the nearest of the decisions
was from going the other way, relative to the mass it was taken on; a decision
on equal weights alone is exact and has margin infinity.
"""
from __future__ import annotations

import numpy as np


def sample_row(logits, u=0.0, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability, margin)."""
    row = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    order = sorted(range(len(row)), key=lambda i: (-row[i], i))
    best = row[order[0]]
    if best == -np.inf:
        return -1, 0.0, np.inf
    if not temperature > 0:
        return order[0], 1.0, np.inf
    if 0 < top_k < len(order):
        order = order[:top_k]
    w = np.array([1.0 if row[i] == best else 0.0 if row[i] == -np.inf else np.exp((row[i] - best) / temperature)
                  for i in order])
    margin = np.inf

    def near(c, target):
        d = np.abs(c - target) / c[-1]
        return np.inf if np.all(w[w > 0] == 1.0) else float(d.min())

    if top_p < 1:
        c = np.cumsum(w)
        target = top_p * c[-1]
        n = 1
        while n < len(w) and c[n - 1] < target:
            n += 1
        margin = min(margin, near(c, target))
        w, order = w[:n], order[:n]
    if min_p > 0:
        kept = [i for i in range(len(w)) if w[i] >= min_p or w[i] == 1.0]
        rest = np.abs(w[w != 1.0] - min_p)
        margin = min(margin, float(rest.min()) if rest.size else np.inf)
        w, order = w[kept], [order[i] for i in kept]
    c = np.cumsum(w)
    target = u * c[-1]
    margin = min(margin, near(c, target)) if 0 < u < 1 else margin
    last = int(np.count_nonzero(w > 0)) - 1
    at = 0
    while at < last and not c[at] > target:
        at += 1
    if not u >= 0:
        at = 0
    return order[at], float(w[at] / c[-1]), margin
