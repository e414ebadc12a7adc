"""Calls of the rotation that share arrays or lie at the ends of what it takes (GB300 only)."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tr():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from free_speculative_decoding_gb300 import build as b
    b.build()
    import free_speculative_decoding_gb300 as m
    return m


@pytest.fixture(autouse=True)
def status_stays_clean(tr):
    yield
    assert tr.tr_get_status() == 0


# One kernel for a sequence's rows, and a plan before it, which advances the lengths first.
@pytest.mark.parametrize("T", [1, 3, 21, 22, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("share", ["pos", "count", "both"])
def test_positions_and_counts_are_the_lengths(tr, T, dtype, share):
    """The cache's lengths as positions, or as counts: their values before the call."""
    B, Hq, Hkv, d, L = 4, 32, 8, 128, [0, 1, 7, T]
    L = [min(x, T) for x in L]
    g = torch.Generator().manual_seed(T)
    qkv = torch.randn(B, T, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    Q, K, V = qkv.split((Hq, Hkv, Hkv), 2)
    rope = tr.Rope(d, (1e4 ** (-torch.arange(0, d, 2).float() / d)).cuda(), q_norm=torch.ones(d, device="cuda"),
                   k_norm=torch.ones(d, device="cuda"))
    scale = torch.full((Hkv,), 0.02, device="cuda") if dtype is torch.float8_e4m3fn else None

    def run(shared):
        Kc, Vc = (torch.zeros(B, Hkv, 2 * T + 8, d, device="cuda").to(dtype) for _ in range(2))
        lengths = torch.tensor(L, dtype=torch.int32, device="cuda")
        cache = tr.KVCache(Kc, Vc, lengths, k_scale=scale, v_scale=scale)
        Qo = torch.full((B, T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        own = lengths if shared else lengths.clone()
        tr.tr_kv_append_rope(Q, K, V, rope, cache, Qo, tr.workspace(tr.tr_kv_append_workspace_bytes(cache)),
                             pos=own if share != "count" else None, count=own if share != "pos" else None)
        return lengths, Qo, Kc.view(torch.uint8), Vc.view(torch.uint8)
    for got, want in zip(run(True), run(False)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T", [1, 40])
def test_frequencies_of_many_turns_a_position(tr, pairs, T):
    """Frequencies from 2^23 to fp32's end, where a step of fp32 is up to 10^30 turns, at far positions.  Below 2^24 the turns
    are known to p (1 + f) 2^-64 only, so the positions are small there.  Tolerance: 10 steps of 2^-24 of the two elements
    (the phase, its rounding, cos and sin, the products), then half a step of fp16."""
    rng = np.random.default_rng(3)
    ends = [2.0 ** 24, 2.0 ** 24 + 2, 2.0 ** 25 - 2, 2.0 ** 87, 2.0 ** 88, 2.0 ** 89 * 1.5, 2.0 ** 127, 3.4028234e38, -2.0 ** 24, -1e9, -3e38]
    f = np.float32(np.concatenate([ends, 2.0 ** rng.uniform(24, 127.9, 32 - len(ends))]))
    far = [1, 0, 3, -5, 10 ** 6, 2 ** 31 - T, -2 ** 31]
    for inv, pos in ((f, far), (np.float32(2.0 ** rng.uniform(22, 24, 32)), [0, 1, 2, 50, 3, 7, 30])):
        x = torch.from_numpy(rng.normal(size=(len(pos), T, 2, 64))).half().cuda()
        y = torch.zeros_like(x)
        tr.tr_qkv_rope(None, x, None, tr.Rope(64, torch.from_numpy(inv).cuda(), pairs=pairs),
                       torch.tensor(pos, dtype=torch.int32, device="cuda"), None, y, None)
        for b, p in enumerate(pos):
            z, size = oracle.rope_rows(x[b].cpu().numpy(), [p + i for i in range(T)], inv, pairs)
            e = 10 * 2.0 ** -24 * size
            assert (np.abs(y[b].cpu().double().numpy() - z) <= e + 2.0 ** -11 * (np.abs(z) + e) + 2.0 ** -25).all(), (p, inv)
