"""RMS norm and position rotation of queries and keys, written out plainly in 64
bits (test infrastructure only)."""
from __future__ import annotations

import numpy as np


def rope_rows(x, pos, inv_freq, pairs=False, weight=None, eps=0.0):
    """Rows x [n, H, d] at the integer positions pos [n]: normed by ``weight`` [d] (None:
    not), then the first 2 * len(inv_freq) elements turned pair by pair by the angle
    pos * inv_freq.  ``pairs``: pair i is (2 i, 2 i + 1), else (i, i + len(inv_freq)).

    Returns the rows and, for the error bounds, each element's |y_i| + |y_j| (the two
    numbers that it is made of; |y_i| where it is not turned)."""
    x = np.asarray(x, np.float64)
    f = np.asarray(inv_freq, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).sum(-1, keepdims=True) / x.shape[-1] + eps) * np.asarray(weight, np.float64)
    out, size = x.copy(), np.abs(x)
    half = len(f)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        angle = np.array([_angle(int(p), f[i]) for p in pos])[:, None]
        c, s = np.cos(angle), np.sin(angle)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return out, size


# 2 pi to 60 digits, as a fraction
_TWO_PI = (6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


def _angle(p, f):
    """p * f less its whole turns, which are dropped in integer arithmetic."""
    num, den = float(f).as_integer_ratio()
    tn, td = _TWO_PI
    n, d = p * num * td, den * tn           # p f / (2 pi) = n / d turns
    n %= d
    return 2.0 * np.pi * (n / d)
