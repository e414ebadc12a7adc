"""The oracle of single-token decoding over a KV cache, pinned against library
routines, closed forms and brute force (no GPU)."""
import itertools

import numpy as np
import pytest
import torch

import oracle


def test_decode_attention_is_library_attention_and_last_row_of_causal():
    rng = np.random.default_rng(1)
    Hkv, G, L, d = 3, 2, 17, 8
    q, k, v = rng.normal(size=(Hkv * G, d)), rng.normal(size=(Hkv, L, d)), rng.normal(size=(Hkv, L, d))
    O, lse, W = oracle.decode_attention(q, k, v, 0.3)
    t = lambda x: torch.from_numpy(x)
    ref = torch.nn.functional.scaled_dot_product_attention(
        t(q)[:, None], t(k).repeat_interleave(G, 0), t(v).repeat_interleave(G, 0), scale=0.3)[:, 0]
    assert np.allclose(O, ref.numpy(), rtol=0, atol=1e-13)
    s = torch.einsum("hd,hld->hl", t(q), t(k).repeat_interleave(G, 0)) * 0.3
    assert np.allclose(lse, torch.logsumexp(s, 1).numpy(), rtol=1e-14)
    assert np.allclose(W, torch.softmax(s, 1).numpy(), rtol=1e-12)


def test_decode_attention_closed_forms():
    rng = np.random.default_rng(2)
    k, v = rng.normal(size=(1, 5, 4)), rng.normal(size=(1, 5, 4))
    O, lse, W = oracle.decode_attention(np.zeros((2, 4)), k, v, 1.0)       # equal logits: the mean
    assert np.allclose(O, v.mean(1)) and np.allclose(lse, np.log(5)) and np.allclose(W, 0.2)
    O, lse, _ = oracle.decode_attention(rng.normal(size=(1, 4)), k[:, :1], v[:, :1], 1.0)   # one row: its value
    assert np.array_equal(O, v[:, 0])
    O, lse, W = oracle.decode_attention(np.ones((1, 4)), k[:, :0], v[:, :0], 1.0)            # no row
    assert not O.any() and np.isneginf(lse).all() and W.shape == (1, 0)
    O, lse, _ = oracle.decode_attention(np.full((1, 4), 1e4), np.stack([k[0], -k[0]])[:1], v, 1.0)
    assert np.isfinite(O).all() and np.isfinite(lse).all()


def test_e4m3_round_is_the_nearest_of_all_values():
    allv = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    grid = np.unique(allv[np.isfinite(allv)])
    assert np.array_equal(oracle.e4m3_round(grid), grid)
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.normal(size=4000) * 10.0 ** rng.integers(-4, 3, 4000), (grid[1:] + grid[:-1]) / 2])
    got = oracle.e4m3_round(x)
    best = np.abs(np.clip(x, -448, 448)[:, None] - grid[None]).min(1)
    assert np.array_equal(np.abs(np.clip(x, -448, 448) - got), best)
    # torch's conversion rounds alike (ties to even) inside the range
    inside = x[np.abs(x) <= 448]
    f = inside.astype(np.float32)
    assert np.array_equal(oracle.e4m3_round(f), torch.from_numpy(f).to(torch.float8_e4m3fn).double().numpy())
    assert np.isnan(oracle.e4m3_round(np.nan)) and oracle.e4m3_round(np.inf) == 448


@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (3, 0), (3, 1), (3, 3), (5, 2)])
def test_evict_keep_by_brute_force(budget, recent):
    """Of all sets allowed, the kept one has the largest ordered scores, then the lowest positions."""
    rng = np.random.default_rng(budget * 10 + recent)
    for _ in range(20):
        s = rng.integers(0, 3, 6).astype(float)
        got = oracle.evict_keep(s, budget, recent)
        prot = set(range(6 - recent, 6))
        sets = [c for c in itertools.combinations(range(6), budget) if prot <= set(c)]
        old = lambda c: [p for p in c if p not in prot]
        best = max(sets, key=lambda c: (sorted((s[p] for p in old(c)), reverse=True), [-p for p in old(c)]))
        assert got == list(best)


def test_evict_keep_special_scores():
    nan, inf = float("nan"), float("inf")
    assert oracle.evict_keep([1, 2], 2, 0) == [0, 1]                     # within the budget
    assert oracle.evict_keep([nan, -inf, nan, 0.0], 2, 0) == [1, 3]
    assert oracle.evict_keep([nan, nan, -inf], 2, 0) == [0, 2]
    assert oracle.evict_keep([0.0, -0.0, 0.0, -0.0], 2, 0) == [0, 1]
    assert oracle.evict_keep([-0.0, 0.0, 1.0], 2, 0) == [0, 2]
    assert oracle.evict_keep([inf, 5, inf, 1, 1], 3, 1) == [0, 2, 4]
    assert oracle.evict_keep([9, 9, 9], 1, 1) == [2]
