"""Calls around the rotation and sampling that are refused on the host (no GPU)."""
import ctypes

import pytest

P = 1 << 20  # an address that is never dereferenced


@pytest.fixture(scope="module")
def tr():
    from free_speculative_decoding_gb300 import build as b
    b.build()
    import free_speculative_decoding_gb300 as m
    m.lib()
    return m


def test_positions_and_counts_that_overlap_the_lengths_in_part(tr):
    B, L = 4, P + 4096
    x = tr.tr_qkv(Q=P, K=P, V=P, type=tr.TR_KV_BF16, B=B, T=5, Hq=8, Hkv=4)
    for name in ("q_stride", "k_stride", "v_stride"):
        setattr(x, name, (ctypes.c_int64 * 3)(5 * 16 * 128, 16 * 128, 128))
    r = tr.tr_rope(d=128, rot=128, pairs=0, inv_freq=P, q_norm=P, k_norm=P, eps=1e-6)
    c = tr.tr_kv_cache(K=P, V=P, type=tr.TR_KV_BF16, B=B, Hkv=4, d=128, L=L, cap=64, block_stride=4 * 64 * 128,
                       head_stride=64 * 128, row_stride=128)

    def call(pos, count):
        return tr.lib().tr_kv_append_rope(ctypes.byref(x), ctypes.byref(r), pos, count, ctypes.byref(c), P, P, 1 << 40, None)
    for off in (4, 8, 12, -4, -8, -12):
        assert call(L + off, None) == call(None, L + off) == call(L, L + off) == tr.TR_E_INVAL, off


@pytest.mark.parametrize("rule", ["temperature", "top_k", "top_p", "min_p"])
def test_rules_without_uniforms(tr, rule):
    """A step that would be greedy all the same; nothing of the state is touched before the refusal."""
    from free_speculative_decoding_gb300.engine import TRState
    state = object.__new__(TRState)
    with pytest.raises(ValueError, match="uniforms"):
        state.finish_decode(None, **{rule: [1]})
