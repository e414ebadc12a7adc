"""What the single-token calls refuse on the host, before the device is touched (no GPU)."""
import ctypes

import pytest
import torch

P = 1 << 20  # an address that is never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def tr():
    from free_speculative_decoding_gb300 import build as b
    b.build()
    import free_speculative_decoding_gb300 as m
    m.lib()
    return m


def cache(tr, **kw):
    c = tr.tr_kv_cache(K=P, V=P, type=tr.TR_KV_BF16, B=2, Hkv=4, d=128, L=P, cap=64, block_stride=4 * 64 * 128,
                       head_stride=64 * 128, row_stride=128, scores=P, scores_ld=64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


PAGED = dict(page_table=P, max_pages=4, page_size=16, num_pages=9, block_stride=4 * 16 * 128, head_stride=16 * 128)
E4M3 = dict(type=2, k_scale=P, v_scale=P)

BAD_CACHES = [  # (fields, refused as)
    (dict(K=None), "INVAL"), (dict(V=None), "INVAL"), (dict(L=None), "INVAL"), (dict(B=0), "INVAL"),
    (dict(Hkv=0), "INVAL"), (dict(type=3), "INVAL"), (dict(d=0), "INVAL"), (dict(d=96), "UNSUPPORTED"),
    (dict(cap=0), "INVAL"), (dict(K=P + 8), "INVAL"), (dict(V=P + 4), "INVAL"),
    (dict(k_scale=P), "INVAL"), (dict(type=2), "INVAL"), (dict(type=2, k_scale=P), "INVAL"),
    (dict(row_stride=120), "INVAL"), (dict(row_stride=132), "INVAL"), (dict(row_stride=0), "INVAL"),
    (dict(head_stride=0), "INVAL"), (dict(head_stride=-8192), "INVAL"), (dict(head_stride=63 * 128), "INVAL"),
    (dict(block_stride=4 * 64 * 128 - 128), "INVAL"), (dict(block_stride=1 << 60), "INVAL"),
    (dict(head_stride=128, row_stride=128), "INVAL"),
    (dict(scores_ld=63), "INVAL"), (dict(scores=P + 2), "INVAL"), (dict(B=1025), "UNSUPPORTED"),
    (dict(PAGED, page_size=24), "UNSUPPORTED"), (dict(PAGED, page_size=0), "INVAL"),
    (dict(PAGED, max_pages=0), "INVAL"), (dict(PAGED, num_pages=0), "INVAL"),
    (dict(PAGED, max_pages=1 << 28, scores=None), "UNSUPPORTED"),
    (dict(PAGED, B=1, Hkv=1, max_pages=(1 << 26) + 1, scores=None), "UNSUPPORTED"),   # 2^30 + 16 positions
    (dict(B=1, Hkv=1, cap=(1 << 30) + 1, scores=None), "UNSUPPORTED"), (dict(PAGED, scores_ld=63), "INVAL"),
]


@pytest.mark.parametrize("fields,code", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(tr, fields, code):
    c = cache(tr, **fields)
    code = getattr(tr, "TR_E_" + code)
    r, lib = ctypes.byref(c), tr.lib()
    assert lib.tr_decode_attn(P, r, 8, 0.1, P, P, 0, P, BIG, None) == code
    assert lib.tr_kv_append(P, P, 1, None, r, P, BIG, None) == code
    assert lib.tr_kv_evict(r, 8, 2, P, BIG, None) == code
    assert lib.tr_decode_attn_workspace_bytes(r, 8, 0) == 0
    assert lib.tr_kv_evict_workspace_bytes(r, 8) == 0


@pytest.mark.parametrize("fields", [dict(L=P + 2), dict(PAGED, page_table=P + 1), dict(E4M3, k_scale=P + 2),
                                    dict(E4M3, v_scale=P + 1)])
def test_misaligned_arrays_are_refused(tr, fields):
    c = cache(tr, **fields)
    r, lib = ctypes.byref(c), tr.lib()
    assert lib.tr_decode_attn(P, r, 8, 0.1, P, P, 0, P, BIG, None) == tr.TR_E_INVAL
    assert lib.tr_kv_append(P, P, 1, None, r, P, BIG, None) == tr.TR_E_INVAL
    assert lib.tr_kv_evict(r, 8, 2, P, BIG, None) == tr.TR_E_INVAL


@pytest.mark.parametrize("fields,code", [
    # B * Hkv * positions is 2^64; strides of the scores whose products pass 2^63
    (dict(PAGED, B=1024, Hkv=1 << 24, max_pages=1 << 10, page_size=1 << 20, num_pages=1, head_stride=1 << 27), "UNSUPPORTED"),
    (dict(scores=P, scores_ld=1 << 62), "INVAL"), (dict(scores=P, scores_ld=(1 << 63) - 1), "INVAL")])
def test_sizes_whose_products_pass_64_bits_are_refused(tr, fields, code):
    c = cache(tr, **{**dict(scores=None), **fields})
    code = getattr(tr, "TR_E_" + code)
    r, lib = ctypes.byref(c), tr.lib()
    assert lib.tr_kv_evict_workspace_bytes(r, 8) == 0
    assert lib.tr_decode_attn_workspace_bytes(r, c.Hkv, 0) == 0
    assert lib.tr_decode_attn(P, r, c.Hkv, 0.1, P, P, 0, P, BIG, None) == code
    assert lib.tr_kv_append(P, P, 1, None, r, P, BIG, None) == code


def test_misaligned_counts_are_refused(tr):
    assert tr.lib().tr_kv_append(P, P, 1, P + 2, ctypes.byref(cache(tr)), P, BIG, None) == tr.TR_E_INVAL


def test_null_cache(tr):
    lib = tr.lib()
    assert lib.tr_decode_attn(P, None, 8, 0.1, P, P, 0, P, BIG, None) == tr.TR_E_INVAL
    assert lib.tr_kv_append(P, P, 1, None, None, P, BIG, None) == tr.TR_E_INVAL
    assert lib.tr_kv_evict(None, 8, 2, P, BIG, None) == tr.TR_E_INVAL


def good(tr):
    """Caches that pass the host checks: what follows them is refused for its own reason."""
    return [cache(tr), cache(tr, **PAGED), cache(tr, **E4M3), cache(tr, **PAGED, **E4M3),
            cache(tr, d=64, row_stride=64), cache(tr, B=1, block_stride=0),
            cache(tr, head_stride=128, row_stride=4 * 128)]  # [B, cap, Hkv, d]


def test_decode_arguments(tr):
    lib, inf, nan = tr.lib(), float("inf"), float("nan")
    for c in good(tr):
        r = ctypes.byref(c)
        need = lib.tr_decode_attn_workspace_bytes(r, 8, 1)
        assert need > 0 and lib.tr_decode_attn_workspace_bytes(r, 8, 0) > 0

        def call(Q=P, Hq=8, scale=0.1, O=P, lse=P, acc=0, ws=P, nb=BIG):
            return lib.tr_decode_attn(Q, r, Hq, scale, O, lse, acc, ws, nb, None)
        for kw in (dict(Q=None), dict(O=None), dict(Q=P + 8), dict(O=P + 4), dict(lse=P + 2), dict(Hq=0),
                   dict(Hq=6), dict(Hq=-4), dict(scale=0.0), dict(scale=-1.0), dict(scale=inf), dict(scale=nan), dict(scale=3e38),
                   dict(ws=None), dict(ws=P + 8), dict(nb=0), dict(acc=1, nb=need - 1)):
            assert call(**kw) == tr.TR_E_INVAL, kw
        assert lib.tr_decode_attn_workspace_bytes(r, 6, 0) == 0
        assert call(Hq=1 << 24) == tr.TR_E_UNSUPPORTED and lib.tr_decode_attn_workspace_bytes(r, 1 << 24, 0) == 0
    c = cache(tr, scores=None)
    assert lib.tr_decode_attn(P, ctypes.byref(c), 8, 0.1, P, P, 1, P, BIG, None) == tr.TR_E_INVAL


def test_append_arguments(tr):
    lib = tr.lib()
    for c in good(tr):
        r = ctypes.byref(c)
        assert lib.tr_kv_append_workspace_bytes(r) >= 4 * c.B
        for args in ((None, P, 1), (P, None, 1), (P + 8, P, 1), (P, P + 8, 1), (P, P, 0), (P, P, -1)):
            assert lib.tr_kv_append(*args, None, r, P, BIG, None) == tr.TR_E_INVAL
        assert lib.tr_kv_append(P, P, 4096, None, r, None, 0, None) == tr.TR_E_INVAL    # needs counters
        assert lib.tr_kv_append(P, P, 4096, None, r, P, 4, None) == tr.TR_E_INVAL


def test_evict_arguments(tr):
    lib = tr.lib()
    for c in good(tr):
        r = ctypes.byref(c)
        need = lib.tr_kv_evict_workspace_bytes(r, 8)
        assert need >= c.B * c.Hkv * 8 * 4 + 4 * c.B
        assert 0 < lib.tr_kv_evict_workspace_bytes(r, 1 << 30) < need + 4096  # a budget that nothing can exceed
        assert lib.tr_kv_evict_workspace_bytes(r, 0) == 0
        for budget, recent, ws, nb in ((0, 0, P, BIG), (-1, 0, P, BIG), (8, -1, P, BIG), (8, 9, P, BIG),
                                       (8, 2, None, BIG), (8, 2, P + 8, BIG), (8, 2, P, need - 1)):
            assert lib.tr_kv_evict(r, budget, recent, ws, nb, None) == tr.TR_E_INVAL
    c = cache(tr, scores=None)
    assert lib.tr_kv_evict(ctypes.byref(c), 8, 2, P, BIG, None) == tr.TR_E_INVAL


def test_binding_refuses_host_tensors(tr):
    L = torch.zeros(2, dtype=torch.int32)
    K = torch.zeros(2, 4, 64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        tr.KVCache(K, K, L)
    with pytest.raises(ValueError, match="bfloat16"):
        tr.KVCache(K.float(), K.float(), L)
    with pytest.raises(ValueError, match="same shape"):
        tr.KVCache(K, K[:, :2], L)
    with pytest.raises(ValueError, match="empty"):
        tr.KVCache(K[:0], K[:0], L)
