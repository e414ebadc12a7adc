"""Sampling one token from a row of logits with temperature, top-k, top-p and min-p,
written out plainly in 64 bits (test infrastructure only)."""
from __future__ import annotations

import math

import numpy as np


def sample_left(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The IDs that the rules leave, ascending, their weights exp((x - max) / T), and how far
    the sum at top-p's edge is from its mark, as a share of the sum (inf without one).
    Nothing is left where every logit is -inf or NaN."""
    x = np.asarray(x, np.float64)
    ids = np.flatnonzero(x > -np.inf)                       # NaN compares false
    if len(ids) == 0:
        return ids, np.zeros(0), np.inf
    m = x[ids].max()
    # falling logits, equal ones by ascending ID
    order = ids[np.lexsort((ids, -x[ids]))]
    if not temperature >= 2.0 ** -126:
        return order[:1], np.ones(1), np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        d = np.where(x[order] == m, 0.0, x[order] - m)
        w = np.where(d == 0.0, 1.0, np.exp(d / temperature))
    if top_k > 0:
        order, w, d = order[:top_k], w[:top_k], d[:top_k]
    margin = np.inf
    if top_p < 1.0:                                          # NaN compares false
        mass, all_ = np.cumsum(w), math.fsum(w)
        mark = max(top_p, 0.0) * all_
        n = max(int(np.searchsorted(mass, mark, side="left")) + 1, 1)
        margin = float(np.abs(mass - mark).min() / all_) if top_p > 0.0 else np.inf
        order, w, d = order[:n], w[:n], d[:n]
    if min_p > 0.0 and temperature < np.inf:
        # by the exponents: a weight just below 1 may round to it
        stay = d >= temperature * math.log(min(min_p, 1.0))
        order, w = order[stay], w[stay]
    at = np.argsort(order)
    return order[at], w[at], margin


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The token drawn by the uniform u, the logarithm of its probability among those left,
    and the distance of the nearest border (of the draw or of top-p's edge)."""
    ids, w, margin = sample_left(x, temperature, top_k, top_p, min_p)
    if len(ids) == 0:
        return -1, -np.inf, np.inf
    u = min(max(u, 0.0), 1.0 - 2.0 ** -24) if u == u else 0.0
    mass, all_ = np.cumsum(w), math.fsum(w)
    k = min(int(np.searchsorted(mass, u * all_, side="right")), len(ids) - 1)
    if len(ids) > 1:
        margin = min(margin, float(np.abs(mass[:-1] - u * all_).min() / all_))
    return int(ids[k]), math.log(w[k] / all_) if w[k] > 0 else -np.inf, margin
