"""What tr_qkv_rope, tr_kv_append_rope and tr_sample refuse on the host, before the device is
touched (no GPU)."""
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


def rows(tr, **kw):
    x = tr.tr_qkv(Q=P, K=P, V=P, type=tr.TR_KV_BF16, B=2, T=5, Hq=8, Hkv=4)
    for name in ("q_stride", "k_stride", "v_stride"):
        setattr(x, name, (ctypes.c_int64 * 3)(5 * 16 * 128, 16 * 128, 128))
    for k, v in kw.items():
        setattr(x, k, (ctypes.c_int64 * 3)(*v) if k.endswith("stride") else v)
    return x


def rope(tr, **kw):
    r = tr.tr_rope(d=128, rot=128, pairs=0, inv_freq=P, q_norm=P, k_norm=P, eps=1e-6)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def cache(tr, **kw):
    c = tr.tr_kv_cache(K=P, V=P, type=tr.TR_KV_BF16, B=2, Hkv=4, d=128, L=P, cap=64, block_stride=4 * 64 * 128,
                       head_stride=64 * 128, row_stride=128, scores=P, scores_ld=64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_ROWS = [
    (dict(B=0), "INVAL"), (dict(T=0), "INVAL"), (dict(T=-3), "INVAL"), (dict(Hq=0), "INVAL"), (dict(Hkv=0), "INVAL"),
    (dict(type=2), "INVAL"), (dict(type=7), "INVAL"), (dict(Q=P + 8), "INVAL"), (dict(K=P + 2), "INVAL"),
    (dict(V=P + 4), "INVAL"), (dict(q_stride=(-8, 2048, 128)), "INVAL"), (dict(k_stride=(8192, 2044, 128)), "INVAL"),
    (dict(v_stride=(8192, 2048, 100)), "INVAL"), (dict(q_stride=(1 << 60, 2048, 128)), "INVAL"),
    (dict(B=1 << 20, T=1 << 12), "UNSUPPORTED"), (dict(B=1 << 15, T=1 << 15), "UNSUPPORTED"), (dict(Hq=(1 << 20) + 1), "UNSUPPORTED"),
    (dict(Hkv=1 << 20), "UNSUPPORTED"),
]
BAD_ROPES = [
    (dict(d=0), "INVAL"), (dict(d=-64), "INVAL"), (dict(rot=-16), "INVAL"), (dict(rot=144), "INVAL"),
    (dict(inv_freq=None), "INVAL"), (dict(inv_freq=P + 2), "INVAL"), (dict(q_norm=P + 1), "INVAL"),
    (dict(k_norm=P + 2), "INVAL"), (dict(eps=-1.0), "INVAL"), (dict(eps=float("nan")), "INVAL"),
    (dict(eps=float("inf")), "INVAL"), (dict(d=96, rot=96), "UNSUPPORTED"), (dict(d=256), "UNSUPPORTED"),
    (dict(rot=20), "UNSUPPORTED"), (dict(rot=8), "UNSUPPORTED"),
]


@pytest.mark.parametrize("bad_rows,bad_rope,code", [(f, {}, c) for f, c in BAD_ROWS] + [({}, f, c) for f, c in BAD_ROPES])
def test_bad_rows_and_rotations(tr, bad_rows, bad_rope, code):
    x, r, c = rows(tr, **bad_rows), rope(tr, **bad_rope), cache(tr)
    code, lib = getattr(tr, "TR_E_" + code), tr.lib()
    assert lib.tr_qkv_rope(ctypes.byref(x), ctypes.byref(r), P, None, P, P, P, None) == code
    assert lib.tr_kv_append_rope(ctypes.byref(x), ctypes.byref(r), P, None, ctypes.byref(c), P, P, BIG, None) == code


def test_rotation_arguments(tr):
    lib, r, x = tr.lib(), ctypes.byref(rope(tr)), rows(tr)
    tree, other = tr.Tree((4, 0, 0, 0, 0), 4), tr.Tree((0,), 4)

    def call(x=x, r=r, pos=P, tree=None, out=(P, P, P)):
        return lib.tr_qkv_rope(ctypes.byref(x) if x is not None else None, r, pos, tree, *out, None)
    for kw in (dict(x=None), dict(r=None), dict(pos=None), dict(pos=P + 2), dict(tree=other.handle),
               dict(out=(None, P, P)), dict(out=(P, None, P)), dict(out=(P, P, None)), dict(out=(P + 8, P, P)),
               dict(out=(P, P + 4, P)), dict(out=(P, P, P + 2)), dict(x=rows(tr, Q=None)), dict(x=rows(tr, V=None)),
               dict(x=rows(tr, Q=None, K=None, V=None), out=(None, None, None))):
        assert call(**kw) == tr.TR_E_INVAL, kw
    del tree


def test_append_rope_arguments(tr):
    lib, r, x, c = tr.lib(), rope(tr), rows(tr), cache(tr)

    def call(x=x, r=r, pos=P, count=P, c=c, Qo=P, ws=P, nb=BIG):
        return lib.tr_kv_append_rope(ctypes.byref(x), ctypes.byref(r), pos, count,
                                     ctypes.byref(c) if c is not None else None, Qo, ws, nb, None)
    for kw in (dict(c=None), dict(pos=P + 1), dict(count=P + 2), dict(Qo=None), dict(Qo=P + 8), dict(ws=None),
               dict(ws=P + 8), dict(nb=15), dict(x=rows(tr, Q=None)), dict(x=rows(tr, K=None)), dict(x=rows(tr, V=None)),
               dict(x=rows(tr, B=1)), dict(x=rows(tr, Hkv=2)), dict(r=rope(tr, d=64, rot=64)),
               dict(x=rows(tr, type=tr.TR_KV_F16)), dict(c=cache(tr, type=tr.TR_KV_F16)),
               dict(c=cache(tr, type=2, k_scale=P, v_scale=P), x=rows(tr, type=tr.TR_KV_F16)),
               dict(c=cache(tr, K=P + 8)), dict(c=cache(tr, cap=0))):
        assert call(**kw) == tr.TR_E_INVAL, kw


def test_sample_arguments(tr):
    lib = tr.lib()

    def call(x=P, ft=tr.TR_F32, rows=4, V=10, ld=10, T=P, k=P, p=P, m=P, U=P, tok=P, lp=P):
        return lib.tr_sample(x, ft, rows, V, ld, T, k, p, m, U, tok, lp, None)
    for kw in (dict(x=None), dict(U=None), dict(tok=None), dict(ft=2), dict(rows=-1), dict(V=0), dict(ld=9), dict(x=P + 2),
               dict(x=P + 1, ft=tr.TR_BF16), dict(T=P + 2), dict(k=P + 1), dict(p=P + 2), dict(m=P + 2), dict(U=P + 1),
               dict(tok=P + 2), dict(lp=P + 2)):
        assert call(**kw) == tr.TR_E_INVAL, kw
    assert call(rows=0, x=None, U=None, tok=None) == tr.TR_OK
    assert call(rows=(1 << 24) + 1) == tr.TR_E_UNSUPPORTED
    assert call(V=(1 << 30) + 1, ld=1 << 31) == tr.TR_E_UNSUPPORTED
    assert call(ld=1 << 60) == tr.TR_E_UNSUPPORTED


def test_binding_refuses(tr):
    f = torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA device"):
        tr.Rope(128, f)
    for kw, what in ((dict(d=96), "d must be"), (dict(d=128, inv_freq=f[:5]), "rot a multiple"),
                     (dict(d=64, inv_freq=f), "at most d"), (dict(d=128, inv_freq=f.double()), "float32"),
                     (dict(d=128, q_norm=f), "q_norm"), (dict(d=128, eps=-1.0), "eps"),
                     (dict(d=128, inv_freq=f[:0]), "inv_freq")):
        with pytest.raises(ValueError, match=what):
            tr.Rope(**kw)
    assert tr.Rope(64).rot == 0
