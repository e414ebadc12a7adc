"""The oracle of the rotation and of sampling, pinned against closed forms, library
routines and brute force (no GPU)."""
import itertools
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle


def test_two_pi_is_right():
    from oracle.rope import _TWO_PI
    n, d = _TWO_PI
    assert float(Fraction(n, d)) == 2 * math.pi
    # Machin: pi = 16 atan(1/5) - 4 atan(1/239), in integers of 10^-70
    one = 10 ** 70

    def atan_inv(k):
        term, total, i = one // k, 0, 1
        while term:
            total += term // i if i % 4 == 1 else -(term // i)
            term //= k * k
            i += 2
        return total
    two_pi = 2 * (16 * atan_inv(5) - 4 * atan_inv(239))
    assert abs(n * 10 ** 10 - two_pi) < 10 ** 11


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance_only(pairs):
    rng = np.random.default_rng(1)
    f = 10.0 ** -rng.uniform(0, 3, 8)
    q, k = rng.normal(size=(1, 2, 24)), rng.normal(size=(1, 2, 24))
    at = lambda x, p: oracle.rope_rows(x, [p], f, pairs)[0]
    assert np.allclose(np.linalg.norm(at(q, 977), axis=-1), np.linalg.norm(q, axis=-1), rtol=1e-13)
    a = (at(q, 100007) * at(k, 100002)).sum(-1)
    b = (at(q, 5) * at(k, 0)).sum(-1)
    assert np.allclose(a, b, rtol=1e-9)
    assert np.array_equal(at(q, 0), q)
    assert np.array_equal(at(q, 3)[..., 16:], q[..., 16:])       # behind the rotated part
    assert np.allclose(at(at(q, 3), -3), q, atol=1e-14)


def test_rotation_is_the_product_of_complex_numbers():
    rng = np.random.default_rng(2)
    x, f = rng.normal(size=(3, 1, 16)), 1e4 ** (-np.arange(8) / 8)
    pos = [0, 7, 12345]
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * np.array(pos)[:, None, None] * f)
    got = oracle.rope_rows(x, pos, f, True)[0]
    assert np.allclose(got[..., 0::2], z.real, atol=1e-12) and np.allclose(got[..., 1::2], z.imag, atol=1e-12)
    # the other layout is the same with its elements in another order
    perm = np.concatenate([np.arange(0, 16, 2), np.arange(1, 16, 2)])
    assert np.array_equal(oracle.rope_rows(x[..., perm], pos, f, False)[0], got[..., perm])


def test_norm_is_the_library_norm():
    rng = np.random.default_rng(3)
    x, w = rng.normal(size=(4, 2, 64)), rng.normal(size=64)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x), (64,), torch.from_numpy(w), eps=1e-3).numpy()
    assert np.allclose(oracle.rope_rows(x, [1] * 4, [], weight=w, eps=1e-3)[0], ref, rtol=1e-13)


def test_far_angles_lose_nothing():
    from oracle.rope import _angle
    f = float(np.float32(0.1))
    for p in (1, 10 ** 5, 2 ** 31 - 1, -(2 ** 31)):
        want = Fraction(p) * Fraction(f)
        from oracle.rope import _TWO_PI
        turns = want / Fraction(*_TWO_PI)
        rest = turns - math.floor(turns)
        assert abs(_angle(p, f) - float(rest) * 2 * math.pi) < 1e-15


def brute_left(x, T, k, p, mp):
    """Every rule by its own words, in fractions of the weights' exact binary values."""
    fin = [v for v in range(len(x)) if x[v] == x[v] and x[v] > -math.inf]
    if not fin:
        return []
    m = max(x[v] for v in fin)
    w = {v: Fraction(math.exp((x[v] - m) / T) if x[v] != m else 1.0) for v in fin}
    if k > 0:
        # of all sets of k tokens the one with the largest logits, then the lowest IDs
        n = min(k, len(fin))
        fin = list(max(itertools.combinations(fin, n),
                       key=lambda c: (sorted((x[v] for v in c), reverse=True), [-v for v in c])))
    if p < 1:
        total = sum(w[v] for v in fin)
        for n in range(1, len(fin) + 1):
            best = max(itertools.combinations(fin, n),
                       key=lambda c: (sorted((x[v] for v in c), reverse=True), [-v for v in c]))
            if sum(w[v] for v in best) >= Fraction(p) * total:
                fin = list(best)
                break
    if mp > 0:
        fin = [v for v in fin if w[v] >= Fraction(min(mp, 1.0))]
    return sorted(fin)


def test_rules_by_brute_force():
    rng = np.random.default_rng(4)
    for _ in range(300):
        x = rng.integers(-3, 3, 7) / 2.0
        x[rng.random(7) < 0.15] = rng.choice([-np.inf, np.nan])
        T, k = rng.choice([0.25, 1.0, 3.0]), int(rng.integers(0, 9))
        p, mp = rng.choice([1.0, 0.31, 0.77, 0.0]), rng.choice([0.0, 0.11, 0.6, 1.5])
        ids, w, _ = oracle.sample_left(x, T, k, p, mp)
        assert list(ids) == brute_left(x, T, k, p, mp)


def test_draw_is_the_inverse_distribution():
    rng = np.random.default_rng(5)
    x = rng.normal(size=40) * 2
    p = torch.softmax(torch.from_numpy(x) / 0.7, 0).numpy()
    n = 20000
    got = np.bincount([oracle.sample(x, (i + 0.5) / n, 0.7)[0] for i in range(n)], minlength=40)
    assert np.abs(got - n * p).max() <= 1.0                      # evenly spaced uniforms: off by less than one
    tok, lp, _ = oracle.sample(x, 0.3, 0.7)
    assert abs(lp - math.log(p[tok])) < 1e-12
    assert oracle.sample([0.0, 0.0], 0.5)[0] == 1 and oracle.sample([0.0, 0.0], 0.5 - 2.0 ** -25)[0] == 0


def test_special_rows():
    inf, nan = np.inf, np.nan
    assert oracle.sample([-inf, nan], 0.5)[:2] == (-1, -inf)
    assert oracle.sample([0.0, 3.0, 3.0], 0.9, temperature=0.0)[:2] == (1, 0.0)
    assert oracle.sample([inf, 5.0, inf], 0.6)[:2] == (2, math.log(0.5))
    assert oracle.sample([nan, 1.0, -inf], 0.999)[0] == 1
    assert oracle.sample([1.0, 2.0, 3.0], nan)[0] == 0 and oracle.sample([1.0, 2.0, 3.0], 7.0)[0] == 2
    assert list(oracle.sample_left([0.0, -5.0, -inf], temperature=inf)[0]) == [0, 1]
