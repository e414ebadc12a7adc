"""Which tokens a draw may give next to a border, pinned by hand (no GPU)."""
import math

import numpy as np
import pytest

import oracle

INF, NAN = math.inf, math.nan
may = oracle.sample_may_draw


def test_only_tokens_that_are_left():
    """At u = 0 every border is near; what the rules leave none of stays out all the same."""
    x = np.array([-INF, -30.0, NAN, 0.0, 1.0, -INF])
    for bad in (0, 2, 5, -1, -7, 6, 10 ** 9):
        assert may(x, bad, 0.0, 1e-8) is None
    assert may(x, 1, 0.0, 1e-8) and may(x, 3, 0.0, 1e-8)      # the first has a weight below the tolerance
    assert may(x, 4, 0.0, 1e-8) is None                        # too far behind
    assert may(x, 3, 0.0, 1e-15) is None
    assert may(x, 1, 0.0, 1e-8, top_k=2) is None and may(x, 3, 0.0, 1e-8, top_k=2)
    assert may(x, 1, 0.0, 1e-8, min_p=1e-3) is None and may(x, 1, 0.0, 1e-8, top_p=0.999) is None
    assert may(x, 4, NAN, 1e-8, temperature=0.0) and may(x, 3, 0.0, 1e-8, temperature=0.0) is None
    assert may([-INF, NAN], -1, 0.5, 1e-8) == (-INF, -INF) and may([-INF, NAN], 0, 0.5, 1e-8) is None
    for T in (1.0, INF):                                       # all the draw is the infinite ones
        assert list(oracle.sample_left([INF, 5.0, INF], temperature=T)[1]) == [1.0, 0.0, 1.0]
        assert oracle.sample([5.0, INF, 5.0], 0.99, temperature=T)[:2] == (1, 0.0)
        assert may([5.0, INF, 5.0], 1, 0.99, 1e-8, temperature=T) and not may([5.0, INF, 5.0], 2, 0.99, 1e-8, temperature=T)
    assert may([INF, 5.0, INF], 2, 0.5 - 1e-9, 1e-8) and may([INF, 5.0, INF], 1, 0.5, 1e-8) is None


def test_stretches_of_the_running_sum():
    x = np.log([1.0, 2.0, 1.0])                                # sums 1/4, 3/4, 1
    for u, want in ((0.0, [0]), (0.24, [0]), (0.2499, [0, 1]), (0.2501, [0, 1]), (0.26, [1]), (0.75, [1, 2]), (1.5, [2])):
        assert [t for t in range(3) if may(x, t, u, 1e-3)] == want, u
    lo, hi = may(x, 1, 0.5, 1e-3)
    assert lo == hi and abs(lo + math.log(2)) < 1e-15


def test_the_edge_of_top_p_within_its_tolerance():
    x = np.log([4.0, 3.0, 2.0, 1.0])                           # of ten; sums 4, 7, 9, 10
    ids = lambda p, u: [t for t in range(4) if may(x, t, u, 1e-3, top_p=p)]
    assert ids(0.65, 0.99) == [1] and ids(0.72, 0.99) == [2]
    assert ids(0.7, 0.99) == [1, 2]                            # two or three are left
    lo, hi = may(x, 0, 0.1, 1e-3, top_p=0.7)
    assert abs(lo - math.log(4 / 9)) < 1e-15 and abs(hi - math.log(4 / 7)) < 1e-15
    # an edge among many small tokens: each of those within the tolerance may be the last
    y = np.concatenate([[0.0], np.full(1000, -10.0)])
    w = math.exp(-10.0)                                        # far above the 2^-24 that u stays below one by
    p = (1 + 500 * w) / (1 + 1000 * w)
    last = [t for t in range(1001) if may(y, t, 1.0, 2.5 * w, top_p=p)]
    assert 500 in last and last == list(range(last[0], last[-1] + 1)) and 490 <= last[0] and last[-1] <= 504


@pytest.mark.parametrize("seed", range(4))
def test_every_exact_draw_may_be_drawn(seed):
    rng = np.random.default_rng(seed)
    for _ in range(300):
        x = rng.integers(-4, 4, 9) / 2.0
        x[rng.random(9) < 0.2] = rng.choice([-INF, NAN])
        kw = dict(temperature=rng.choice([0.0, 0.5, 1.0, INF]), top_k=int(rng.integers(0, 6)),
                  top_p=rng.choice([1.0, 0.9, 0.3, 0.0, NAN]), min_p=rng.choice([0.0, 0.2, 1.0, 2.0]))
        u = rng.choice([0.0, 0.25, 0.5, rng.random(), 1.0])
        t, lp, margin = oracle.sample(x, u, **kw)
        got = may(x, t, u, 1e-12, **kw)
        assert got is not None and got[0] - 1e-11 <= lp <= got[1] + 1e-11, (x, kw, u)
        if margin > 1e-9:
            assert [v for v in range(-1, 10) if may(x, v, u, 1e-12, **kw)] == [t], (x, kw, u)
