"""Norms and position rotation of queries and keys on the GPU against the 64-bit oracle, into
dense rows and into a KV cache (GB300 only).

Tolerance, from the arithmetic: u = 2^-24 is half a step of fp32.  The sum of a row's d
squares runs as chains of at most d adds and multiplications (each off by u), the square root halves
that error, rsqrtf adds two steps, two more products follow: a normed element is off by at
most (d / 2 + 8) u, relative: 72 u < 2^-17 at d = 128.  The angle is known to p (1 + f) 2^-64 turns
and to 2^-32 of one, rounded to fp32 as half turns (at most 1: off by u, pi u in radians); cos and sin add two steps
of at most 2u each: under 8 u absolute.  A rotated element is a sum of two products, so it is off by at
most (2^-17 + 10 u) (|y_i| + |y_j|) < 2^-16 (|y_i| + |y_j|), without a norm 10 u < 2^-20
of it, and then by half a step of the output's type, relative, or of its smallest step."""
import numpy as np
import pytest
import torch

import oracle
import synth

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
# half a step relative, half the smallest step
HALF = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25), "e4m3": (2.0 ** -4, 2.0 ** -10)}


@pytest.fixture(scope="module")
def tr():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from free_speculative_decoding_gb300 import build as b
    b.build()
    import free_speculative_decoding_gb300 as m
    assert torch.cuda.get_device_capability() == (10, 3)
    return m


@pytest.fixture(autouse=True)
def status_stays_clean(tr):
    yield
    assert tr.tr_get_status() == 0


def f64(x):
    return x.detach().cpu().double().numpy()


def bound(size, z, type, norm, scale=1.0):
    rel, least = HALF[type]
    e = (2.0 ** -16 if norm else 2.0 ** -20) * size
    return e + rel * (np.abs(z) + e) + least * scale


class Case:
    """A rope with its inputs: Q, K, V as views of one projection's output."""

    def __init__(self, tr, type="bf16", B=2, T=3, Hq=4, Hkv=2, d=128, rot=None, pairs=False, norm=True, seed=0, eps=1e-6,
                 base=1e4):
        g = torch.Generator().manual_seed(seed)
        self.type, self.wide = type, torch.float16 if type == "f16" else torch.bfloat16
        self.rot = d if rot is None else rot
        self.pairs, self.eps = pairs, eps
        qkv = (torch.randn(B, T, Hq + 2 * Hkv, d, generator=g) * torch.exp(torch.randn(1, 1, Hq + 2 * Hkv, 1, generator=g)))
        self.qkv = qkv.to(self.wide).cuda()
        self.Q, self.K, self.V = self.qkv[:, :, :Hq], self.qkv[:, :, Hq:Hq + Hkv], self.qkv[:, :, Hq + Hkv:]
        self.B, self.T, self.Hq, self.Hkv, self.d = B, T, Hq, Hkv, d
        self.inv = (base ** (-torch.arange(0, self.rot, 2).float() / max(self.rot, 1))) if self.rot else None
        self.wq, self.wk = (1 + 0.5 * torch.randn(2, d, generator=g)).unbind(0) if norm else (None, None)
        cu = lambda t: None if t is None else t.cuda()
        self.rope = tr.Rope(d, cu(self.inv), pairs=pairs, q_norm=cu(self.wq), k_norm=cu(self.wk), eps=eps)

    def expect(self, x, weight, pos):
        """The oracle's rows of x [n, H, d] and the bound of their error before the output's rounding."""
        f = [] if self.inv is None else self.inv.numpy()
        return oracle.rope_rows(f64(x), pos, f, self.pairs, None if weight is None else weight.numpy(), np.float32(self.eps))

    def check_rows(self, got, x, weight, pos):
        want, size = self.expect(x, weight, pos)
        t = "f16" if self.type == "f16" else "bf16"
        assert (np.abs(f64(got) - want) <= bound(size, want, t, weight is not None)).all()

    def check_dense(self, out, pos):
        for b in range(self.B):
            self.check_rows(out[0][b], self.Q[b], self.wq, pos[b])
            self.check_rows(out[1][b], self.K[b], self.wk, pos[b])
        assert torch.equal(out[2].view(torch.int16), self.V.contiguous().view(torch.int16))

    def outputs(self):
        e = lambda H: torch.full((self.B, self.T, H, self.d), 7.0, dtype=self.wide, device="cuda")
        return e(self.Hq), e(self.Hkv), e(self.Hkv)

    def run(self, tr, pos, tree=None):
        out = self.outputs()
        tr.tr_qkv_rope(self.Q, self.K, self.V, self.rope, torch.tensor(pos, dtype=torch.int32, device="cuda"), *out,
                       tree=tree)
        return out


@pytest.mark.parametrize("type", ["bf16", "f16"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 0), (128, 128), (128, 96), (128, 64), (128, 16)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_types_and_layouts(tr, type, d, rot, pairs, norm):
    c = Case(tr, type, d=d, rot=rot, pairs=pairs, norm=norm)
    out = c.run(tr, [0, 1000])
    c.check_dense(out, [[0, 1, 2], [1000, 1001, 1002]])


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 32, 32), (3, 1, 15, 5), (1, 33, 7, 7), (2, 129, 40, 1), (5, 7, 3, 3),
                                        (70, 2, 12, 4), (1, 700, 32, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_rope_sizes(tr, B, T, Hq, Hkv, d):
    c = Case(tr, "bf16", B, T, Hq, Hkv, d, norm=B % 2 == 0, pairs=T % 2 == 0)
    pos = [17 * b for b in range(B)]
    c.check_dense(c.run(tr, pos), [[p + i for i in range(T)] for p in pos])


@pytest.mark.parametrize("counts", [synth.TREE_T80, synth.TREE_T128, (0,), (2, 1, 0, 0), (1, 1, 1, 0)])
def test_rope_tree_positions(tr, counts):
    tree = tr.Tree(counts, 8)
    c = Case(tr, "bf16", 2, tree.N, 4, 2)
    c.check_dense(c.run(tr, [5, 3000], tree), [[p + x for x in tree.depth] for p in (5, 3000)])


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_far_positions(tr, pairs):
    """Positions to the ends of 32 bits, frequencies of long contexts and above one: the angle in
    fp32 would be off by whole turns."""
    c = Case(tr, "f16", 6, 2, 2, 1, pairs=pairs, norm=False, base=1e7)
    pos = [1 << 20, (1 << 22) + 3, 10 ** 9, (1 << 31) - 1, -5, -(1 << 31)]
    c.check_dense(c.run(tr, pos), [[p, p + 1] for p in pos])
    c.inv = c.inv * 3.7
    c.rope = tr.Rope(c.d, c.inv.cuda(), pairs=pairs)
    c.check_dense(c.run(tr, pos), [[p, p + 1] for p in pos])


def test_rope_strides_and_in_place(tr):
    c = Case(tr, "bf16", 3, 5, 4, 4, 128)
    want = c.run(tr, [4, 5, 6])
    # [B, H, T, d] memory, every second row of a longer buffer, heads of one row shared by all (a stride of 0)
    for make in (lambda x: x.transpose(1, 2).contiguous().transpose(1, 2),
                 lambda x: torch.stack((x, x), 2).flatten(1, 2)[:, ::2],
                 lambda x: torch.cat((x, x), 3)[..., :128]):
        out = c.outputs()
        pos = torch.tensor([4, 5, 6], dtype=torch.int32, device="cuda")
        tr.tr_qkv_rope(make(c.Q), make(c.K), make(c.V), c.rope, pos, *out)
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    one = c.K[:, :, :1].expand(3, 5, 4, 128)
    out = c.outputs()
    tr.tr_qkv_rope(None, one, None, c.rope, pos, None, out[1], None)
    assert torch.equal(out[1], want[1][:, :, :1].expand_as(out[1]))
    # each output may be its input
    q, k, v = c.Q.contiguous(), c.K.contiguous(), c.V.contiguous()
    tr.tr_qkv_rope(q, k, v, c.rope, pos, q, k, v)
    assert all(torch.equal(x, y) for x, y in zip((q, k, v), want))
    # one of the three alone
    for i, (x, name) in enumerate(((c.Q, "Q"), (c.K, "K"), (c.V, "V"))):
        ins, outs, fresh = [None] * 3, [None] * 3, c.outputs()
        ins[i], outs[i] = x, fresh[i]
        tr.tr_qkv_rope(*ins, c.rope, pos, *outs)
        assert torch.equal(fresh[i], want[i]), name


def test_rope_special_values_stay_in_their_head(tr):
    c = Case(tr, "bf16", 2, 4, 4, 2, 128, norm=True)
    want = c.run(tr, [3, 9])
    c.qkv[0, 1, 2, 5] = float("nan")
    c.qkv[1, 3, 5, 100] = float("inf")      # a key
    c.qkv[1, 2, 7, 1] = float("-inf")       # a value
    c.qkv[0, 0, 1] = 0.0                    # a row of zeros: 0 / sqrt(eps)
    got = c.run(tr, [3, 9])
    mask = torch.ones(2, 4, 4, dtype=torch.bool, device="cuda")
    mask[0, 1, 2] = mask[0, 0, 1] = False
    assert torch.equal(got[0][mask], want[0][mask]) and torch.isnan(got[0][0, 1, 2]).all() and not got[0][0, 0, 1].any()
    mask = torch.ones(2, 4, 2, dtype=torch.bool, device="cuda")
    mask[1, 3, 1] = False
    assert torch.equal(got[1][mask], want[1][mask])
    assert torch.isinf(got[2][1, 2, 1, 1])


def test_rope_wide_range_of_magnitudes(tr):
    """Rows of 2^-60 to 2^60 (their squares fit fp32), with and without a norm."""
    for norm in (False, True):
        c = Case(tr, "bf16", 1, 61, 2, 1, 128, norm=norm, eps=0.0)
        c.qkv *= (2.0 ** torch.arange(-60, 61, 2, device="cuda").double()).view(1, 61, 1, 1).to(torch.bfloat16)
        c.check_dense(c.run(tr, [7]), [[7 + i for i in range(61)]])


# ---------------------------------------------------------------------------
# into a cache
# ---------------------------------------------------------------------------

class Pool:
    """A cache for the rows of a Case, filled with NaN, and what it holds."""

    def __init__(self, tr, c, layout, lengths, scores=True, seed=1):
        g = torch.Generator().manual_seed(seed)
        dt = TYPES[c.type]
        B = c.B
        cap = max(lengths) + c.T + 3
        bits = dict(dtype=torch.uint8) if c.type == "e4m3" else dict(dtype=torch.int16)
        nan = 0x7F if c.type == "e4m3" else 0x7FFF
        self.pt = None
        if layout == "dense":
            shape = (B, c.Hkv, cap, c.d)
        else:
            mp = -(-cap // layout)
            P = B * mp + 3
            self.pt = torch.randperm(P, generator=g)[:B * mp].view(B, mp).to(torch.int32).cuda()
            cap = mp * layout
            shape = (P, c.Hkv, layout, c.d)
        self.K, self.V = (torch.full(shape, nan, device="cuda", **bits).view(dt) for _ in range(2))
        self.L = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.ks = self.vs = None
        if c.type == "e4m3":
            self.ks, self.vs = ((0.01 + 0.1 * torch.rand(c.Hkv, generator=g)).cuda() for _ in range(2))
        self.scores = torch.ones(B, c.Hkv, cap, device="cuda") if scores else None
        self.cache = tr.KVCache(self.K, self.V, self.L, page_table=self.pt, scores=self.scores, k_scale=self.ks,
                                v_scale=self.vs)
        self.ws = tr.workspace(tr.tr_kv_append_workspace_bytes(self.cache))
        self.layout = layout

    def rows(self, x, b, n):
        """[n, Hkv, d] of sequence b, as stored."""
        raw = x.view(torch.uint8) if x.element_size() == 1 else x
        if self.pt is None:
            r = raw[b, :, :n]
        else:
            r = raw[self.pt[b].long()].transpose(1, 2).reshape(-1, raw.shape[1], raw.shape[3])[:n].transpose(0, 1)
        return r.transpose(0, 1).contiguous().view(x.dtype)


def check_append(tr, c, layout, lengths, counts=None, pos=None):
    p = Pool(tr, c, layout, lengths)
    plain = Pool(tr, c, layout, lengths)
    Qo = torch.full((c.B, c.T, c.Hq, c.d), 7.0, dtype=c.wide, device="cuda")
    t32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")
    tr.tr_kv_append_rope(c.Q, c.K, c.V, c.rope, p.cache, Qo, p.ws, pos=t32(pos), count=t32(counts))
    tr.tr_kv_append(c.K.contiguous(), c.V.contiguous(), plain.cache, plain.ws, count=t32(counts))
    assert torch.equal(p.L, plain.L) and torch.equal(p.scores, plain.scores)
    raw = lambda x: x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int16)
    assert torch.equal(raw(p.V), raw(plain.V))                       # values go as tr_kv_append takes them
    nan = lambda x: torch.isnan(x.float())
    assert torch.equal(nan(p.K), nan(plain.K))                       # and keys to the same places
    for b in range(c.B):
        n = c.T if counts is None else counts[b]
        if n == 0:
            continue
        first = lengths[b] if pos is None else pos[b]
        at = [first + i for i in range(n)]
        c.check_rows(Qo[b, :n], c.Q[b, :n], c.wq, at)
        want, size = c.expect(c.K[b, :n], c.wk, at)
        got = f64(p.rows(p.K, b, lengths[b] + n)[lengths[b]:].float())
        if p.ks is None:
            assert (np.abs(got - want) <= bound(size, want, c.type, c.wk is not None)).all()
        else:
            s = f64(p.ks)[None, :, None]
            clip = np.clip(want, -448 * s, 448 * s)
            assert (np.abs(got * s - clip) <= bound(size, clip, "e4m3", c.wk is not None, s)).all()
        assert (Qo[b, n:] == 7.0).all()
    return p, Qo


@pytest.mark.parametrize("type", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 32)])
@pytest.mark.parametrize("layout", ["dense", 1, 16, 64])
@pytest.mark.parametrize("T", [1, 2, 40])
def test_append_rope(tr, type, d, rot, layout, T):
    c = Case(tr, type, 3, T, 6, 3, d, rot=rot, pairs=layout == 16, norm=T != 2)
    check_append(tr, c, layout, [0, 5, 130])
    check_append(tr, c, layout, [0, 5, 130], counts=[0, T, T // 2], pos=[9, 1 << 20, 0])


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 32, 32), (1, 1, 1, 1), (64, 1, 32, 8), (1, 3, 160, 32), (2, 300, 12, 4), (1, 1, 71, 71),
                                        (3, 9, 5, 5), (1024, 1, 2, 1)])
@pytest.mark.parametrize("type", ["bf16", "e4m3"])
def test_append_rope_sizes(tr, B, T, Hq, Hkv, type):
    c = Case(tr, type, B, T, Hq, Hkv, 128)
    check_append(tr, c, 16, [(37 * b) % 101 for b in range(B)])


def test_append_rope_is_the_two_calls(tr):
    """Into 16-bit caches the same bits as tr_qkv_rope and then tr_kv_append; without queries too."""
    for type, T in (("bf16", 1), ("f16", 1), ("bf16", 50)):
        c = Case(tr, type, 3, T, 8, 4, 128)
        L = [7, 0, 64]
        p, Qo = check_append(tr, c, 64, L)
        out = c.run(tr, L)
        two = Pool(tr, c, 64, L)
        tr.tr_kv_append(out[1], out[2], two.cache, two.ws)
        bits = lambda x: x.view(torch.int16)
        assert torch.equal(Qo, out[0]) and torch.equal(bits(p.K), bits(two.K)) and torch.equal(bits(p.V), bits(two.V))
        no_q = Pool(tr, c, 64, L)
        tr.tr_kv_append_rope(None, c.K, c.V, c.rope, no_q.cache, None, no_q.ws)
        assert torch.equal(bits(no_q.K), bits(two.K)) and torch.equal(no_q.L, two.L)
        q = c.Q.contiguous()
        own = Pool(tr, c, 64, L)
        tr.tr_kv_append_rope(q, c.K, c.V, c.rope, own.cache, q, own.ws)      # in place
        assert torch.equal(q, Qo)


@pytest.mark.parametrize("T", [1, 3, 200])
def test_append_rope_bad_inputs_leave_the_sequence(tr, T):
    c = Case(tr, "bf16", 5, T, 4, 2, 128)
    L = [3, 4, 0, 10, 20]
    p = Pool(tr, c, 16, L)
    p.L[0] = -1                                   # outside the cache
    p.L[1] = p.cache.cap - T + 1                  # full
    p.pt[2, 0] = 1 << 30                          # points nowhere
    before = [x.clone() for x in (p.K, p.V, p.L, p.scores)]
    Qo = torch.full((5, T, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    tr.tr_kv_append_rope(c.Q, c.K, c.V, c.rope, p.cache, Qo, p.ws)
    assert tr.tr_get_status() == tr.TR_DEV_BAD_LENGTH | tr.TR_DEV_CACHE_FULL | tr.TR_DEV_BAD_PAGE
    assert torch.equal(p.L[:3], before[2][:3]) and (p.L[3:] == torch.tensor([10 + T, 20 + T], device="cuda")).all()
    assert (Qo[:3] == 7.0).all() and not (Qo[3:] == 7.0).all()
    assert torch.equal(p.scores[:3], before[3][:3])
    for pages in (p.pt[1].long(), p.pt[0].long(), p.pt[2, 1:].long()):
        assert torch.isnan(p.K[pages].float()).all() and torch.isnan(p.V[pages].float()).all()
    for b in (3, 4):
        c.check_rows(p.rows(p.K, b, L[b] + T)[L[b]:], c.K[b], c.wk, [L[b] + i for i in range(T)])
    count = torch.tensor([-1, T + 1, 0, 0, 0], dtype=torch.int32, device="cuda")
    p2 = Pool(tr, c, 16, L)
    tr.tr_kv_append_rope(c.Q, c.K, c.V, c.rope, p2.cache, Qo, p2.ws, count=count)
    assert tr.tr_get_status() == tr.TR_DEV_BAD_LENGTH and p2.L.tolist() == L


def test_rope_offsets_past_32_bits(tr):
    """Rows whose elements lie past 2^31 from the first, in and out, and a cache as large."""
    d, H, T = 128, 1, 3
    x = torch.zeros(2, T, (1 << 31) // (T * d) + 5, d, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.empty(2, T, H, d, device="cuda").normal_(generator=g).bfloat16()
    x[:, :, -1:] = k
    inv = 1e4 ** (-torch.arange(0, d, 2).float() / d)
    rope = tr.Rope(d, inv.cuda())
    pos = torch.tensor([3, 8], dtype=torch.int32, device="cuda")
    out, want = torch.empty_like(k), torch.empty_like(k)
    tr.tr_qkv_rope(None, x[:, :, -1:], None, rope, pos, None, out, None)
    tr.tr_qkv_rope(None, k, None, rope, pos, None, want, None)
    assert torch.equal(out, want)
    del x
    # the output's last rows lie past 2^31 elements: one row repeated by a stride of 0
    T = (1 << 31) // (64 * d) + 2
    big = k[:1, :1].expand(1, T, 64, d)
    y = torch.empty(1, T, 64, d, dtype=torch.bfloat16, device="cuda")
    tr.tr_qkv_rope(None, big, None, rope, pos[:1], None, y, None)
    one, last = k[:1, :1].contiguous(), torch.empty(1, 1, H, d, dtype=torch.bfloat16, device="cuda")
    tr.tr_qkv_rope(None, one, None, rope, pos[:1] + (T - 1), None, last, None)
    assert torch.equal(y[0, -1], last[0, 0].expand(64, d))


def test_rope_in_a_graph_on_another_stream(tr):
    """Captured once, replayed with other inputs, positions, counts and lengths; two calls of one graph share the workspace."""
    c = Case(tr, "bf16", 3, 4, 8, 4, 128)
    p = Pool(tr, c, 16, [5, 0, 20])
    pos = torch.tensor([5, 70, 1 << 18], dtype=torch.int32, device="cuda")
    count = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    Qo, out = c.outputs()[0], c.outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            tr.tr_kv_append_rope(c.Q, c.K, c.V, c.rope, p.cache, Qo, p.ws, pos=pos, count=count)
            tr.tr_kv_append_rope(c.Q, c.K, c.V, c.rope, p.cache, Qo, p.ws, pos=pos, count=count)
            tr.tr_qkv_rope(c.Q, c.K, c.V, c.rope, pos, *out)
        for rep in range(3):
            c.qkv.mul_(-0.5)
            pos.add_(3)
            if rep:
                count.copy_(torch.tensor([rep, 1, 0]))
            n, before = count.tolist(), p.L.tolist()
            g.replay()
            s.synchronize()
            assert p.L.tolist() == [x + 2 * y for x, y in zip(before, n)]
            at = pos.tolist()
            c.check_dense(out, [[x + i for i in range(4)] for x in at])
            for b in range(3):
                for call in range(2):
                    lo = before[b] + call * n[b]
                    c.check_rows(p.rows(p.K, b, lo + n[b])[lo:], c.K[b, :n[b]], c.wk, [at[b] + i for i in range(n[b])])
    torch.cuda.current_stream().wait_stream(s)


def test_rope_binding_refuses(tr):
    c = Case(tr, "bf16", 2, 3, 4, 2, 128)
    out = c.outputs()
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    p = Pool(tr, c, 16, [1, 2])

    def rope(Q=c.Q, K=c.K, V=c.V, rope=c.rope, pos=pos, out=out, tree=None):
        tr.tr_qkv_rope(Q, K, V, rope, pos, *out, tree=tree)

    def append(Q=c.Q, K=c.K, V=c.V, rope=c.rope, Qo=out[0], cache=p.cache, ws=p.ws, **kw):
        tr.tr_kv_append_rope(Q, K, V, rope, cache, Qo, ws, **kw)
    rope()
    append()
    bad = [dict(Q=c.Q.float()), dict(K=c.K.half()), dict(Q=c.Q[:1]), dict(K=c.K[:, :2]), dict(V=c.V[..., :64]),
           dict(V=c.V[:, :, :1]), dict(Q=c.Q.cpu()), dict(Q=c.Q[0]), dict(Q=c.Q.transpose(2, 3).contiguous().transpose(2, 3)),
           dict(rope=tr.Rope(64)), dict(pos=pos.long()), dict(pos=pos[:1]), dict(pos=pos.cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            rope(**kw)
        if "pos" not in kw or True:
            with pytest.raises(ValueError):
                append(**kw)
    for kw in (dict(out=(None,) + out[1:]), dict(Q=None), dict(out=(out[1], out[1], out[2])), dict(tree=tr.Tree((0,), 2)),
               dict(Q=None, K=None, V=None, out=(None,) * 3), dict(out=(out[0].float(),) + out[1:]),
               dict(out=(c.Q,) + out[1:])):
        with pytest.raises(ValueError):
            rope(**kw)
    for kw in (dict(K=None), dict(Qo=None), dict(count=pos[:1]), dict(count=pos.long()), dict(ws=p.ws.int()), dict(Qo=out[1]),
               dict(K=c.K[:, :, :1], V=c.V[:, :, :1])):
        with pytest.raises(ValueError):
            append(**kw)
    with pytest.raises(tr.TRError):
        rope(pos=None)
    with pytest.raises(tr.TRError):
        append(ws=p.ws[:8])
    off = torch.empty(c.Q.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 3, 4, 128)
    with pytest.raises(tr.TRError):
        rope(Q=off)                                                      # not 16-byte aligned
    assert p.L.tolist() == [4, 5]


def test_rope_norms_of_one_kind_and_unaligned_arrays(tr):
    """A norm of the queries or the keys alone, weights and frequencies at any 4 bytes, and no rotation without positions."""
    for type, d, pairs in (("bf16", 128, False), ("f16", 64, True)):
        for q, k in ((True, False), (False, True), (True, True)):
            c = Case(tr, type, 3, 21, 8, 2, d, pairs=pairs)
            off = lambda t: torch.cat([t.new_zeros(1), t]).cuda()[1:]
            c.wq, c.wk = c.wq if q else None, c.wk if k else None
            c.rope = tr.Rope(d, off(c.inv), pairs=pairs, q_norm=None if c.wq is None else off(c.wq),
                             k_norm=None if c.wk is None else off(c.wk), eps=c.eps)
            c.check_dense(c.run(tr, [0, 7, 4000]), [[p + i for i in range(21)] for p in (0, 7, 4000)])
            check_append(tr, c, 16, [0, 3, 77], counts=[21, 0, 5])
        c = Case(tr, type, 2, 5, 4, 4, d, rot=0)
        out = c.outputs()
        tr.tr_qkv_rope(c.Q, c.K, c.V, c.rope, None, *out)
        c.check_dense(out, [[0] * 5] * 2)


# 6 tasks a token (12 groups): up to 128 tasks a cluster takes a sequence, more go by a plan to all SMs.
@pytest.mark.parametrize("T", [21, 22, 85, 86])
@pytest.mark.parametrize("type", ["bf16", "f16", "e4m3"])
def test_append_rope_on_both_sides_of_the_plan(tr, T, type):
    c = Case(tr, type, 4, T, 32, 8, 128)
    check_append(tr, c, 16, [0, 5, 130, 64])
    check_append(tr, c, "dense", [0, 5, 130, 64], counts=[0, T, 1, T - 1], pos=[9, 1 << 20, 0, 3])


# Shares of a token: few tokens, some, as many as warps, and many (two shares behind a norm).
@pytest.mark.parametrize("T", [3, 30, 200, 607, 609, 5000])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (9, 2)])
def test_rope_shares(tr, T, Hq, Hkv):
    c = Case(tr, "bf16", 4, T, Hq, Hkv, 128, seed=T)
    pos = [0, 11, 1 << 16, 5]
    c.check_dense(c.run(tr, pos), [[p + i for i in range(T)] for p in pos])


def test_rope_on_two_streams_at_once(tr):
    """Calls of both kinds under way at a time, each with its own workspace, give what they give alone."""
    sizes = [("bf16", 2, 700, 8, 2), ("f16", 8, 3, 32, 8), ("bf16", 1, 1, 32, 32), ("e4m3", 3, 200, 12, 4)]
    cases = [Case(tr, t, B, T, Hq, Hkv, 128, seed=i) for i, (t, B, T, Hq, Hkv) in enumerate(sizes)]
    raw = lambda x: x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int16)

    def run(c, pool, pos, out):
        tr.tr_kv_append_rope(c.Q, c.K, c.V, c.rope, pool.cache, out[3], pool.ws)
        tr.tr_qkv_rope(c.Q, c.K, c.V, c.rope, pos, *out[:3])
    state = lambda c: (Pool(tr, c, 16, [5 * b for b in range(c.B)]),
                       torch.arange(c.B, dtype=torch.int32, device="cuda"), c.outputs() + c.outputs()[:1])
    alone = [state(c) for c in cases]
    for c, s in zip(cases, alone):
        run(c, *s)
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for rep in range(3):
        both = [state(c) for c in cases]
        torch.cuda.synchronize()
        for i, (c, s) in enumerate(zip(cases, both)):
            with torch.cuda.stream(streams[(i + rep) % len(cases)]):
                run(c, *s)
        torch.cuda.synchronize()
        for (p, _, out), (p2, _, out2) in zip(alone, both):
            assert torch.equal(p.L, p2.L) and torch.equal(raw(p.K), raw(p2.K)) and torch.equal(raw(p.V), raw(p2.V))
            assert all(torch.equal(raw(x), raw(y)) for x, y in zip(out, out2))


@pytest.mark.parametrize("T", [1, 5, 60])
@pytest.mark.parametrize("type", ["bf16", "e4m3"])
def test_append_rope_into_strided_caches(tr, T, type):
    """Pages of [position, K or V, head, d] in one tensor, and a slice of a larger dense cache: what lies between the rows
    stays as it was, and the rows are those of a contiguous cache."""
    c = Case(tr, type, 3, T, 6, 3, 64)
    L, page = [4, 0, 33], 16
    plain = Pool(tr, c, page, L)
    Qo = c.outputs()[0]
    tr.tr_kv_append_rope(c.Q, c.K, c.V, c.rope, plain.cache, Qo, plain.ws)
    raw = lambda x: x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int16)
    mark = 0x7F if type == "e4m3" else 0x7FFF
    n, dt = plain.K.shape[0], plain.K.dtype
    bits = raw(plain.K).dtype
    both = torch.full((n, page, 2, 4, 64), mark, dtype=bits, device="cuda")
    K, V = (both[:, :, i, :3].view(dt).transpose(1, 2) for i in range(2))
    wide = torch.full((2, 5, 7, 4 * page * 2, 64), mark, dtype=bits, device="cuda")
    Kd, Vd = (wide[i, 1:4, 2:5].view(dt) for i in range(2))
    for K, V, pt in ((K, V, plain.pt), (Kd, Vd, None)):
        L2 = torch.tensor(L, dtype=torch.int32, device="cuda")
        cache = tr.KVCache(K, V, L2, page_table=pt, scores=torch.ones(3, 3, 200, device="cuda"), k_scale=plain.ks, v_scale=plain.vs)
        Q2 = torch.full_like(Qo, 7.0)
        tr.tr_kv_append_rope(c.Q, c.K, c.V, c.rope, cache, Q2, tr.workspace(tr.tr_kv_append_workspace_bytes(cache)))
        assert torch.equal(Q2, Qo) and torch.equal(L2, plain.L)
        assert all((cache.scores[b, :, L[b]:L[b] + T] == 0).all() and cache.scores[b].sum() == 3 * (200 - T) for b in range(3))
        if pt is not None:
            assert torch.equal(raw(K), raw(plain.K)) and torch.equal(raw(V), raw(plain.V))
        else:
            for b in range(3):
                for own, want in ((K, plain.K), (V, plain.V)):
                    assert torch.equal(raw(own[b, :, L[b]:L[b] + T].transpose(0, 1).contiguous()),
                                       raw(plain.rows(want, b, L[b] + T)[L[b]:].contiguous()))
    assert (both[:, :, :, 3] == mark).all()
    assert (wide[:, 0] == mark).all() and (wide[:, 4] == mark).all() and (wide[:, :, :2] == mark).all() and (wide[:, :, 5:] == mark).all()
    for b in range(3):
        assert (wide[:, 1 + b, :, :L[b]] == mark).all() and (wide[:, 1 + b, :, L[b] + T:] == mark).all()
