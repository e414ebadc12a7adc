"""A decoding loop as a program runs it, with the rotation and the sampling in it: tree steps
(rotate, verify, finish) and steps without a draft (decode, finish_decode with uniforms) on one
TRState, evictions between them, against the oracle (GB300 only)."""
import numpy as np
import pytest
import torch

import oracle
import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tr():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from free_speculative_decoding_gb300 import build as b
    b.build()
    import free_speculative_decoding_gb300 as m
    return m


def rotated(x, pos, inv, weight):
    """What the oracle gives for rows x [n, H, d], and how far bf16 ones may be from it (the bound of
    tests/test_gpu_rope.py)."""
    z, size = oracle.rope_rows(x, pos, inv, False, weight, np.float32(1e-6))
    return z, 2.0 ** -16 * size * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(z)


@pytest.mark.parametrize("budget", [0, 100])
def test_engine_with_rope_and_sampling(tr, budget):
    from free_speculative_decoding_gb300.engine import TRState
    from gpu_util import ATTN_TOL, gpu_start, oracle_states, rows_rel_err, target_fn
    from synth import device as sd

    w = synth.WORKLOADS["tiny"].scaled(prefix=(100, 140), B=2, Hq=8, Hkv=4, V=5000, steps=24)
    tree, plan = tr.Tree(w.child_counts, w.K), oracle.TreePlan(w.child_counts, w.K)
    g = torch.Generator().manual_seed(1)
    inv = 1e4 ** (-torch.arange(0, w.d, 2).float() / w.d)
    wq, wk = 1 + 0.3 * torch.randn(w.d, generator=g), 1 + 0.3 * torch.randn(w.d, generator=g)
    rope = tr.Rope(w.d, inv.cuda(), q_norm=wq.cuda(), k_norm=wk.cuda())
    inv, wq, wk = inv.numpy(), wq.numpy(), wk.numpy()
    st = TRState(tree, w.B, w.V, Hq=w.Hq, Hkv=w.Hkv, d=w.d, cap=w.capacity(), single_token=True, budget=budget,
                 recent=20 if budget else 0, rope=rope)
    sd.fill_cache(w, st)
    gpu_start(w, st)
    states, target = oracle_states(w), target_fn(w)
    tgt, logits1 = sd.DeviceTarget(w, tree), torch.empty(w.B, w.V, device="cuda")
    pos = [x.L for x in states]
    rng, f64 = np.random.default_rng(2), lambda t: t.cpu().double().numpy()
    T, k, p, mp = (torch.tensor(v, device="cuda") for v in ([0.9, 0.5], [40, 0], [0.95, 0.9], [0.0, 0.02]))
    k, evicted, drawn = k.int(), 0, 0
    for s in range(w.steps):
        q, kt, vt = sd.step_qkv(w, s, tree.N)
        qkv = torch.cat((q, kt, vt), 2)                       # as one projection leaves them
        q, kt, vt = qkv.split((w.Hq, w.Hkv, w.Hkv), 2)
        plain = s % 3 != 0
        if plain:
            tr.trsyn_logits(w.seed, st.tree1, st.root.unsqueeze(1), st.L, logits1)
            U = torch.tensor(rng.random(w.B), dtype=torch.float32, device="cuda")
            before_kv = [(x.kc.copy(), x.vc.copy()) for x in states]
            O = f64(st.decode(q[:, 0], kt[:, 0], vt[:, 0]))
            st.finish_decode(logits1, U, temperature=T, top_k=k, top_p=p, min_p=mp)
            for b, x in enumerate(states):
                zq, eq = rotated(f64(q[b, :1]), [pos[b]], inv, wq)
                zk, ek = rotated(f64(kt[b, :1]), [pos[b]], inv, wk)
                Q1, K1 = f64(st.Q1[b:b + 1]), f64(st.Kc[b, :, x.L])[None]
                assert (np.abs(Q1 - zq) <= eq).all() and (np.abs(K1 - zk) <= ek).all()
                x.kc, x.vc = before_kv[b]
                x.kc[:, x.L], x.vc[:, x.L] = K1[0], f64(vt[b, 0])
                x.L += 1
                ref, _, _ = oracle.decode_attention(Q1[0], x.kc[:, :x.L], x.vc[:, :x.L], w.d ** -0.5)
                assert rows_rel_err(O[b][None], ref[None]) <= ATTN_TOL
                row = target(b, np.array([x.L - 1]), np.array([x.root]))[0]
                x.M[x.root] = oracle.topk_rows(row[None], w.K)[0][0]
                t, _, margin = oracle.sample(row, float(U[b]), float(T[b]), int(k[b]), float(p[b]), float(mp[b]))
                assert margin > 1e-7
                drawn += t != x.M[x.root][0]
                x.root = t
                pos[b] += 1
                assert st.committed1[b].tolist() == [t] and st.acc_len[b].item() == 0
        else:
            Q, Kt, Vt = st.rotate(q, kt, vt)
            for b, x in enumerate(states):
                at = [pos[b] + d for d in plan.depth]
                zq, eq = rotated(f64(q[b]), at, inv, wq)
                zk, ek = rotated(f64(kt[b]), at, inv, wk)
                assert (np.abs(f64(Q[b]) - zq) <= eq).all() and (np.abs(f64(Kt[b]) - zk) <= ek).all()
            got = f64(st.verify(Q, Kt, Vt))
            rows, recs = (f64(Q), f64(Kt), f64(Vt)), {}
            oracle.tr_loop(plan, states, target, 1, w.K, qkv=lambda _: rows, scale=w.d ** -0.5,
                           on_step=lambda _, b, rec: recs.__setitem__(b, rec))
            st.finish(logits=tgt.logits_for(st), Kt=Kt, Vt=Vt)
            for b in range(w.B):
                assert rows_rel_err(got[b], recs[b]["O"]) <= ATTN_TOL
                pos[b] += recs[b]["acc_len"] + 1
        for b, x in enumerate(states):
            assert st.root[b].item() == x.root and st.L[b].item() == x.L and st.pos[b].item() == pos[b]
            assert np.array_equal(st.M[b].cpu().numpy(), x.M)
            assert np.array_equal(st.tree_tok[b].cpu().numpy(), oracle.retrieve(x.M, x.root, plan))
        if budget and s % 5 == 4:
            sc = st.scores.cpu().numpy()
            st.evict()
            for b, x in enumerate(states):
                if x.L > budget:
                    evicted += 1
                    for h in range(w.Hkv):
                        keep = oracle.evict_keep(sc[b, h, :x.L], budget, 20)
                        for t in (x.kc, x.vc):
                            t[h, :budget] = t[h, keep]
                    x.L = budget
    assert drawn >= 4 and (not budget or (evicted >= 4 and all(a > x.L for a, x in zip(pos, states))))
    assert tr.tr_get_status() == 0
    with pytest.raises(ValueError, match="rope"):
        TRState(tree, 1, 100, rope=rope)
    with pytest.raises(ValueError, match="rope"):
        TRState(tree, 1, 100, Hq=2, Hkv=1, d=128, cap=64, rope=tr.Rope(64))


def test_rope_and_sampling_steps_in_a_graph(tr):
    """A whole step without a draft, captured and replayed, ends where the eager one does."""
    from free_speculative_decoding_gb300.engine import TRState
    from gpu_util import gpu_start
    from synth import device as sd

    w = synth.WORKLOADS["tiny"].scaled(prefix=(100, 140), B=2, Hq=8, Hkv=4, V=5000, steps=8)
    tree = tr.Tree(w.child_counts, w.K)
    rope = tr.Rope(w.d, (1e4 ** (-torch.arange(0, w.d, 2).float() / w.d)).cuda())
    st = TRState(tree, w.B, w.V, Hq=w.Hq, Hkv=w.Hkv, d=w.d, cap=w.capacity(), single_token=True, rope=rope)
    sd.fill_cache(w, st)
    gpu_start(w, st)
    names = ("M", "L", "root", "tree_tok", "Kc", "Vc", "pos", "acc_len", "committed1")
    start = {k: getattr(st, k).clone() for k in names}
    q, kt, vt = sd.step_qkv(w, 0, tree.N)
    logits = torch.randn(w.B, w.V, device="cuda") * 3
    tree_logits = torch.randn(w.B * tree.N, w.V, device="cuda")
    U, T, p = torch.tensor([0.3, 0.8], device="cuda"), torch.tensor([0.7, 1.1], device="cuda"), torch.tensor([0.9, 0.5], device="cuda")

    def steps():
        for _ in range(2):
            st.decode(q[:, 0], kt[:, 0], vt[:, 0])
            st.finish_decode(logits, U, temperature=T, top_p=p)
            Q, Kt, Vt = st.rotate(q, kt, vt)
            st.verify(Q, Kt, Vt)
            st.finish(logits=tree_logits, Kt=Kt, Vt=Vt)
    steps()
    torch.cuda.synchronize()
    want = {k: getattr(st, k).clone() for k in names}
    O = st.O.clone(), st.O1.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for _ in range(2):
        for k in names:
            getattr(st, k).copy_(start[k])
        graph.replay()
        torch.cuda.synchronize()
        for k in names:
            assert torch.equal(getattr(st, k), want[k]), k
        assert torch.equal(st.O, O[0]) and torch.equal(st.O1, O[1])
    assert tr.tr_get_status() == 0
