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
        w = np.where(d == 0.0, 1.0, np.where(d == -np.inf, 0.0, np.exp(d / temperature)))
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


def sample_may_draw(x, token, u, tol, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Whether arithmetic whose sums are off by up to ``tol`` of them may draw ``token`` by the uniform
    u: the token has to be one that the rules leave, top-p's edge lying anywhere within tol of its
    mark, and u times the sum within tol of its stretch of the running sum over ascending IDs.

    Returns the least and the greatest logarithm of its probability as the edge moves, None where the
    token may not be drawn.  A row in which nothing is left may only give -1."""
    token, x = int(token), np.asarray(x, np.float64)
    ids, w, _ = sample_left(x, temperature, top_k)           # ascending IDs
    if len(ids) == 0:
        return (-np.inf, -np.inf) if token == -1 else None
    k = int(np.searchsorted(ids, token))
    if k == len(ids) or ids[k] != token or w[k] == 0.0:      # out of range, masked, NaN, behind the k-th, no weight
        return None
    u = min(max(u, 0.0), 1.0 - 2.0 ** -24) if u == u else 0.0
    order, whole = np.lexsort((ids, -x[ids])), math.fsum(w)
    lo = hi = len(ids)                                       # how many of `order` top-p leaves
    if top_p < 1.0:
        p, mass = max(top_p, 0.0), np.cumsum(w[order])
        lo, hi = (min(max(int(np.searchsorted(mass, mark * whole, side="left")) + 1, 1), len(ids))
                  for mark in (p - tol, p + tol if p else 0.0))
    stay = np.ones(len(ids), bool)
    if min_p > 0.0 and temperature < np.inf and len(ids) > 1:
        with np.errstate(invalid="ignore"):
            stay = (x[ids] == x[ids].max()) | (x[ids] - x[ids].max() >= temperature * math.log(min(min_p, 1.0)))
    rank = np.empty(len(ids), int)
    rank[order] = np.arange(len(ids))
    found = []
    # the sums that edges from lo to hi - 1 leave differ by less than 2 tol of the whole: lo stands for them
    for n, reach, slack in ((lo, max(lo, hi - 1), 2 * tol * whole if hi > lo else 0.0), (hi, hi, 0.0)):
        left = stay & (rank < n)
        sum_ = math.fsum(w[left])
        before = math.fsum(w[:k][left[:k]])
        after = before + (w[k] if left[k] else 0.0)
        slack += tol * sum_
        if stay[k] and rank[k] < reach and before - slack <= u * sum_ <= after + slack:
            found.append(math.log(w[k] / sum_))
    return (min(found), max(found)) if found else None


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
