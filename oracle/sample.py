"""The token sampler, stated plainly in f64 (test infrastructure; see the package docstring).

Tokens in order of falling logit, lowest index first on ties; top-k keeps the first k of the order,
top-p the shortest prefix of those whose weight reaches p times theirs, min-p the tokens with
l >= max + T ln(min_p); the draw is the first index at which the running weight of the kept tokens
exceeds u times their whole weight. T = 0: the arg max.
"""
from __future__ import annotations

import math

import numpy as np


def kept(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(indices kept, rising; their weights exp((l - max) / T))."""
    x = np.asarray(logits, np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    if len(order) == 0:
        return order, np.zeros(0)
    top = x[order[0]]
    w = np.exp((x[order] - top) / temperature)
    n = len(order) if top_k <= 0 else min(len(order), int(top_k))
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w[:n])])
        n = max(1, int(np.count_nonzero(before[:-1] < float(top_p) * before[-1])))
    if min_p > 0:
        n = min(n, int(np.count_nonzero(x[order] >= top + (temperature * math.log(min_p) if min_p < 1 else 0.0))))
    index = np.sort(order[:n])
    return index, np.exp((x[index] - top) / temperature)


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability, distance of u from the nearest border of its share): -1 and 0 for a row with no token."""
    if temperature == 0:
        x = np.asarray(logits, np.float64)
        x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
        return (int(np.argmax(x)), 1.0, 1.0) if x.max() > -np.inf else (-1, 0.0, 1.0)
    index, w = kept(logits, temperature, top_k, top_p, min_p)
    if len(index) == 0:
        return -1, 0.0, 1.0
    total = np.cumsum(w)
    n = min(int(np.searchsorted(total, u * total[-1], side="right")), len(index) - 1)
    share = total / total[-1]
    gap = min(share[n] - u, u - (share[n - 1] if n else -1.0))
    return int(index[n]), float(w[n] / total[-1]), float(gap)
