"""Single-token decoding over a KV cache, written out plainly in 64 bits (test
infrastructure only): attention of one new token, the rounding of an 8-bit
cache, and which rows an eviction by accumulated attention weight keeps."""
from __future__ import annotations

import numpy as np


def decode_attention(q, k, v, scale):
    """One new token of one sequence: q [Hq, d] over k, v [Hkv, L, d].

    Query head h reads KV head h // (Hq / Hkv).  Returns O [Hq, d], the log of
    each head's softmax denominator [Hq] and the weights [Hq, L].  Without any
    row O is 0 and the log-sum is -inf."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    Hq, Hkv, L = q.shape[0], k.shape[0], k.shape[1]
    O, lse, W = np.zeros((Hq, v.shape[2])), np.full(Hq, -np.inf), np.zeros((Hq, L))
    if L == 0:
        return O, lse, W
    for h in range(Hq):
        g = h // (Hq // Hkv)
        s = scale * (k[g] @ q[h])
        m = s.max()
        e = np.exp(s - m)
        W[h] = e / e.sum()
        O[h] = W[h] @ v[g]
        lse[h] = m + np.log(e.sum())
    return O, lse, W


def e4m3_round(x):
    """x rounded to the nearest e4m3 value (sign, four exponent bits with bias 7,
    three fraction bits; no infinities, largest 448), ties to the even fraction,
    larger values clamped, NaN kept."""
    x = np.clip(np.asarray(x, np.float64), -448.0, 448.0)
    _, e = np.frexp(x)                                # |x| in [2^(e-1), 2^e)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)       # below 2^-6 the step stays
    return np.rint(x / step) * step


def evict_keep(scores, budget, recent):
    """Positions that one KV head of a sequence of len(scores) rows keeps, ascending:
    the last `recent`, and of those before them the budget - recent with the
    largest scores (ties to the lower position, -0 equal to +0, NaN below -inf)."""
    L = len(scores)
    if L <= budget:
        return list(range(L))
    old = [(float(s), p) for p, s in enumerate(scores[:L - recent])]
    # NaN is the only value that differs from itself: its group sorts behind all others
    best = sorted(old, key=lambda t: (t[0] != t[0], -t[0] if t[0] == t[0] else 0.0, t[1]))[:budget - recent]
    return sorted(p for _, p in best) + list(range(L - recent, L))
