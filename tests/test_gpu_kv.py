"""Single-token decoding over a KV cache on the GPU against the 64-bit oracle:
attention of one new token, appending rows, evicting rows, and the three
together (GB300 only).

Tolerance of the attention, from the arithmetic: u = 2^-24 is half a step of
fp32.  Products of two 16-bit (or 8-bit) numbers are exact in fp32; a logit is a
sum of d of them, each add off by at most a whole step (2u) where the matrix
unit truncates, then a handful of fp32 roundings, so it is off by at most
delta = (d + 8) * 2u * A with A = scale * max_p sum_i |q_i k_pi|.  A weight is
off by delta (plus 2^-22 of the hardware's 2^x), relative.  Sums over the rows
run as chains of at most L / 8 + 64 adds.  So every output element is within
eps = 2 * (delta + 2^-22 + (L / 8 + 64) * 2u) of sum_p w_p |v_p|, and lse within
delta + 2^-22 + (L / 8 + 64) * 2u + 4u |lse|.  Where the weights are multiplied as
two fp16 parts (fp16 and 8-bit rows) each is also off by up to half of fp16's
smallest step, 2^-25, in a scale in which the largest is at least 2^7: by 2^-32 of
the largest, which the sum of weights is no smaller than.  That adds 2^-32 sum_p |v_p|
(seen where the rows of all larger weights hold a 0 in some column).  The three
bf16 parts have fp32's range: 2^-126 in the place of 2^-32."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


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


def raw(x):
    return x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int16)


class Made:
    """A cache of random rows in a given layout and its contents on the host.

    layout: "dense" [B, Hkv, cap, d]; "dense_nhd" the same stored [B, cap, Hkv, d];
    "wide" dense rows inside wider ones (a stride of 2 d); an int n: pages of n
    rows in random order; "nhd<n>": pages stored [n, Hkv, d].  What no row
    occupies is NaN, unused page table entries point nowhere."""

    def __init__(self, tr, rng, type, layout, lengths, Hkv, d, extra=0, scores=True, spare_pages=3):
        dt = TYPES[type]
        self.type, self.Hkv, self.d, self.lengths = type, Hkv, d, list(lengths)
        B = len(lengths)
        cap = max(max(lengths) + extra, 1)
        g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
        ps, nhd = None, False
        if isinstance(layout, int):
            ps = layout
        elif layout.startswith("nhd"):
            ps, nhd = int(layout[3:]), True
        self.ps = ps
        if ps:
            mp = -(-cap // ps) + 1
            cap = mp * ps
            need = [-(-(n + extra) // ps) for n in lengths]
            P = sum(need) + spare_pages
            perm = torch.randperm(P, generator=g).to(torch.int32)
            pt = torch.full((B, mp), -1, dtype=torch.int32)
            pt[:, 1::2] = 1 << 30
            at = 0
            for b, n in enumerate(need):
                pt[b, :n] = perm[at:at + n]
                at += n
            self.pt_host, self.pt = pt, pt.cuda()
            shape = (P, Hkv, ps, d)
        else:
            self.pt, shape = None, (B, Hkv, cap, d)
        self.cap = cap

        def alloc():
            fill = 0x7F if type == "e4m3" else 0x7FFF
            it = torch.uint8 if type == "e4m3" else torch.int16
            if nhd or layout == "dense_nhd":
                x = torch.full((shape[0], shape[2], shape[1], d), fill, dtype=it, device="cuda").transpose(1, 2)
            elif layout == "wide":
                x = torch.full(shape[:3] + (2 * d,), fill, dtype=it, device="cuda")[..., d:]
            else:
                x = torch.full(shape, fill, dtype=it, device="cuda")
            return x.view(dt)
        self.K, self.V = alloc(), alloc()
        self.ks = self.vs = None
        if type == "e4m3":
            self.ks = (0.01 + 0.02 * torch.rand(Hkv, generator=g)).cuda()
            self.vs = (0.01 + 0.02 * torch.rand(Hkv, generator=g)).cuda()
        self.rows_k, self.rows_v = [], []  # per sequence [Hkv, L, d] on the host, as stored
        for b, n in enumerate(lengths):
            for x, keep in ((self.K, self.rows_k), (self.V, self.rows_v)):
                r = torch.randn(Hkv, n, d, generator=g)
                r = (r * 60).clamp(-448, 448).to(dt) if type == "e4m3" else r.to(dt)
                keep.append(r)
                self.put(x, b, r)
        self.L = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.scores = None
        if scores:
            self.scores = torch.randn(B, Hkv, cap + 3, generator=g).abs().cuda()
        self.tr = tr
        self.cache = tr.KVCache(self.K, self.V, self.L, page_table=self.pt, scores=self.scores, k_scale=self.ks,
                                v_scale=self.vs)
        self.g = g

    def put(self, x, b, r):
        n = r.shape[1]
        x, r = raw(x), raw(r).cuda()
        if self.pt is None:
            x[b, :, :n] = r
        else:
            for i in range(0, n, self.ps):
                m = min(self.ps, n - i)
                x[int(self.pt_host[b, i // self.ps]), :, :m] = r[:, i:i + m]

    def get(self, x, b, n):
        """Rows [0, n) of sequence b as stored, on the host."""
        if self.pt is None:
            return x[b, :, :n].cpu()
        if n == 0:
            return x[0, :, :0].cpu()
        pages = self.pt_host[b, :-(-n // self.ps)].tolist()
        return torch.cat([raw(x)[p].cpu() for p in pages], 1)[:, :n].view(x.dtype)

    def f64(self, rows, scale):
        r = rows.double().numpy()
        return r if scale is None else r * scale.cpu().double().numpy()[:, None, None]

    def queries(self, Hq, factor=1.0):
        B = len(self.lengths)
        return (torch.randn(B, Hq, self.d, generator=self.g) * factor).to(self.cache.row_dtype)

    def attend(self, Q, scale, accumulate=False, ws=None, lse=True):
        tr, B, Hq = self.tr, len(self.lengths), Q.shape[1]
        O = torch.full((B, Hq, self.d), float("nan"), device="cuda")
        lse = torch.full((B, Hq), float("nan"), device="cuda") if lse else None
        if ws is None:  # its contents do not matter
            ws = torch.full((tr.tr_decode_attn_workspace_bytes(self.cache, Hq, accumulate),), 0xFF, dtype=torch.uint8,
                            device="cuda")
        tr.tr_decode_attn(Q.cuda() if not Q.is_cuda else Q, self.cache, O, scale, ws, lse=lse, accumulate=accumulate)
        return O, lse

    def check(self, Q, scale, O, lse, scores_before=None):
        """Every output within the bound that the module's docstring derives."""
        O, Q = O.double().cpu().numpy(), Q.cpu()
        lse = None if lse is None else lse.double().cpu().numpy()
        G = Q.shape[1] // self.Hkv
        for b, n in enumerate(self.lengths):
            k, v = self.f64(self.rows_k[b], self.ks), self.f64(self.rows_v[b], self.vs)
            q = Q[b].double().numpy()
            Or, lr, W = oracle.decode_attention(q, k, v, scale)
            if n == 0:
                assert not O[b].any(), "O of an empty sequence"
                assert lse is None or np.isneginf(lse[b]).all()
            else:
                A = scale * max((np.abs(q[h]) * np.abs(k[h // G])).sum(1).max() for h in range(len(q)))
                delta = (self.d + 8) * 2 * U * A
                one = delta + 2.0 ** -22 + (n / 8 + 64) * 2 * U
                mag = np.stack([W[h] @ np.abs(v[h // G]) for h in range(len(q))])
                least = 2.0 ** (-126 if self.type == "bf16" else -32)
                bound = 2 * one * mag + least * np.stack([np.abs(v[h // G]).sum(0) for h in range(len(q))])
                err = np.abs(O[b] - Or)
                assert (err <= bound).all(), "seq %d (%d rows): %.3g of the bound" % (b, n, (err / bound).max())
                if lse is not None:
                    assert (np.abs(lse[b] - lr) <= one + 4 * U * np.abs(lr)).all()
            if scores_before is not None:
                before = scores_before[b].cpu()
                after = self.scores[b].cpu()
                assert torch.equal(after[:, n:], before[:, n:]), "scores behind the last row"
                if n:
                    add = W.reshape(self.Hkv, G, n).sum(1)
                    ref = before[:, :n].double().numpy() + add
                    tol = 2 * one * add + (G + 2) * U * ref
                    assert (np.abs(after[:, :n].double().numpy() - ref) <= tol).all()


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257]


# ----------------------------------------------------------------------------
# attention of one new token
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("type", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["dense", 16, 64])
@pytest.mark.parametrize("Hkv,G", [(2, 1), (3, 4), (1, 8), (2, 9)])
def test_decode_edge_lengths(tr, type, d, layout, Hkv, G):
    """Lengths around every tile edge, empty sequences among them; all types, head sizes and group kinds."""
    c = Made(tr, np.random.default_rng(d + G), type, layout, EDGES, Hkv, d)
    Q = c.queries(Hkv * G, 2.0)
    before = c.scores.clone()
    O, lse = c.attend(Q, d ** -0.5, accumulate=True)
    c.check(Q, d ** -0.5, O, lse, before)


@pytest.mark.parametrize("type", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv,G", [(3, 4), (1, 8), (2, 9), (1, 40)])
@pytest.mark.parametrize("reach", [1 << 14, 1 << 18])
def test_decode_edge_lengths_in_large_tables(tr, type, d, Hkv, G, reach):
    """The same lengths in caches that could hold far more: what is launched goes by the table's reach (ranges over
    all pairs, of 8 and of 12 warps, instead of one cluster for each)."""
    c = Made(tr, np.random.default_rng(d + G + 1), type, 16, EDGES, Hkv, d, scores=False)
    wide = torch.full((len(EDGES), reach // 16), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.pt.shape[1]] = c.pt
    c.scores = torch.rand(len(EDGES), Hkv, reach, device="cuda")
    c.cache = tr.KVCache(c.K, c.V, c.L, page_table=wide, scores=c.scores, k_scale=c.ks, v_scale=c.vs)
    Q = c.queries(Hkv * G, 2.0)
    before = c.scores.clone()
    O, lse = c.attend(Q, d ** -0.5, accumulate=True)
    c.check(Q, d ** -0.5, O, lse, before)
    first = c.scores.clone()
    c.scores.copy_(before)
    O2, lse2 = c.attend(Q, d ** -0.5, accumulate=True)
    assert torch.equal(O, O2) and torch.equal(lse, lse2) and torch.equal(c.scores, first)


@pytest.mark.parametrize("layout", ["dense_nhd", "wide", 1, 2, 8, 32, 256, 1024, "nhd4", "nhd16", "nhd64"])
@pytest.mark.parametrize("type", ["bf16", "e4m3"])
def test_decode_layouts(tr, layout, type):
    c = Made(tr, np.random.default_rng(7), type, layout, [300, 0, 1, 77, 513, 256], 2, 128)
    Q = c.queries(6, 2.0)
    before = c.scores.clone()
    O, lse = c.attend(Q, 0.1, accumulate=True)
    c.check(Q, 0.1, O, lse, before)
    O2, _ = c.attend(Q, 0.1, lse=False)  # without the optional parts: the same output
    assert torch.equal(O, O2)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 8, 10, 15, 16, 17, 24, 33, 71, 160])
def test_decode_group_sizes(tr, G):
    c = Made(tr, np.random.default_rng(G), "bf16", 16, [90, 1, 700, 0, 33], 1 if G > 40 else 3, 128)
    Q = c.queries(c.Hkv * G, 1.5)
    before = c.scores.clone()
    O, lse = c.attend(Q, 0.09, accumulate=True)
    c.check(Q, 0.09, O, lse, before)


@pytest.mark.parametrize("type,lengths,Hkv,G,layout", [
    ("bf16", [40000], 2, 4, "dense"), ("bf16", [9001, 3, 0, 20000, 1], 1, 12, 128), ("e4m3", [30000, 517], 2, 8, 16),
    ("f16", [12345] * 3, 4, 1, "nhd64"), ("bf16", [2500] * 40, 4, 2, 64), ("bf16", list(range(0, 600)), 1, 1, 16)])
def test_decode_long_and_many(tr, type, lengths, Hkv, G, layout):
    """Sequences cut into many parts, and more sequences than parts."""
    c = Made(tr, np.random.default_rng(len(lengths)), type, layout, lengths, Hkv, 128)
    Q = c.queries(Hkv * G, 2.0)
    before = c.scores.clone()
    O, lse = c.attend(Q, 128 ** -0.5, accumulate=True)
    c.check(Q, 128 ** -0.5, O, lse, before)


def test_decode_most_sequences(tr):
    c = Made(tr, np.random.default_rng(3), "bf16", 16, [(7 * b) % 40 for b in range(1024)], 1, 64)
    Q = c.queries(2)
    O, lse = c.attend(Q, 0.125)
    c.check(Q, 0.125, O, lse)


@pytest.mark.parametrize("type", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("G", [1, 8, 16])
def test_decode_extreme_logits(tr, type, G):
    """Logits of many thousands (one row takes all), all equal ones, and a maximum that keeps rising along the rows."""
    c = Made(tr, np.random.default_rng(5), type, 16, [600, 600, 600, 600], 1, 128)
    Q = c.queries(G, 1.0)
    Q[0] *= 300.0
    Q[1] = 0.0
    for b, order in ((2, 1), (3, -1)):  # rising, falling
        r = torch.linspace(-order, order, 600).reshape(1, 600, 1) * (100.0 if type == "e4m3" else 6.0)
        c.rows_k[b] = (r.expand(1, 600, 128)).to(TYPES[type]).contiguous()
        c.put(c.K, b, c.rows_k[b])
        Q[b] = Q[b].abs() * 0.5
    before = c.scores.clone()
    O, lse = c.attend(Q, 0.5, accumulate=True)
    assert torch.isfinite(O).all() and torch.isfinite(lse).all()
    c.check(Q, 0.5, O, lse, before)


@pytest.mark.parametrize("type", ["bf16", "f16", "e4m3"])
def test_decode_zero_columns_under_the_peak(tr, type):
    """The rows of nearly all weight hold 0 in half of the columns: what is left there comes from weights of 2^-20
    to 2^-50 of the largest, and is right as far as these are kept."""
    n = 40
    c = Made(tr, np.random.default_rng(16), type, 16, [n, n], 1, 128)
    for b in range(2):
        k, v = torch.zeros(1, n, 128), torch.randn(1, n, 128, generator=c.g) * (30 if type == "e4m3" else 1)
        k[0, :, 0] = -torch.arange(n) * (8.0 if type == "e4m3" else 0.5)
        v[0, :10 + 20 * b, ::2] = 0.0
        c.rows_k[b], c.rows_v[b] = k.to(TYPES[type]), v.to(TYPES[type])
        c.put(c.K, b, c.rows_k[b])
        c.put(c.V, b, c.rows_v[b])
    Q = torch.zeros(2, 3, 128, dtype=c.cache.row_dtype)
    Q[..., 0] = torch.tensor([1.0, 2.0, 4.0])
    before = c.scores.clone()
    scale = 4.0 if type == "e4m3" else 1.0
    O, lse = c.attend(Q, scale, accumulate=True)
    c.check(Q, scale, O, lse, before)


@pytest.mark.parametrize("type", ["bf16", "f16"])
def test_decode_flat_tail_behind_one_peak(tr, type):
    """One row holds most of the weight and 20000 share the rest, each far below it: their sum still counts."""
    n = 20001
    c = Made(tr, np.random.default_rng(6), type, 64, [n], 1, 128)
    k = torch.zeros(1, n, 128)
    k[0, 7, 0] = 12.0  # weight e^12 against 20000
    k[0, :, 1] = torch.randn(n, generator=c.g) * 0.01
    v = torch.ones(1, n, 128)
    v[0, 7] = -1.0
    c.rows_k[0], c.rows_v[0] = k.to(TYPES[type]), v.to(TYPES[type])
    c.put(c.K, 0, c.rows_k[0])
    c.put(c.V, 0, c.rows_v[0])
    Q = torch.zeros(1, 2, 128, dtype=c.cache.row_dtype)
    Q[..., 0] = 1.0
    Q[..., 1] = 1.0
    before = c.scores.clone()
    O, lse = c.attend(Q, 1.0, accumulate=True)
    c.check(Q, 1.0, O, lse, before)


def test_decode_small_magnitudes_e4m3(tr):
    """Queries far from 1 (they are narrowed inside for an 8-bit cache) and rows of the smallest 8-bit values."""
    for factor in (1e-30, 1e-6, 1e6, 1e30):
        c = Made(tr, np.random.default_rng(8), "e4m3", 16, [100, 40], 2, 128)
        for b in range(2):
            c.rows_k[b] = (torch.randn(2, c.lengths[b], 128, generator=c.g) * 0.01).to(TYPES["e4m3"])
            c.put(c.K, b, c.rows_k[b])
        Q = c.queries(8, factor)
        scale = min(1.0 / factor, 1e30)
        O, lse = c.attend(Q, scale)
        c.check(Q, scale, O, lse)


def widened(tr, c, reach):
    """The same cache under a page table that could hold `reach` rows a sequence (pages of 16)."""
    wide = torch.full((len(c.lengths), reach // 16), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.pt.shape[1]] = c.pt
    c.scores = torch.rand(len(c.lengths), c.Hkv, reach, device="cuda")
    c.cache = tr.KVCache(c.K, c.V, c.L, page_table=wide, scores=c.scores, k_scale=c.ks, v_scale=c.vs)


@pytest.mark.parametrize("reach", [0, 1 << 14, 1 << 18])   # one cluster for each pair, ranges of 8 and 12 warps
@pytest.mark.parametrize("d,G", [(64, 4), (128, 8), (128, 12)])
def test_decode_e4m3_scales_at_and_below_zero(tr, reach, d, G):
    """A head whose scale is 0 (or so small that its logits vanish) weighs all rows alike; a negative scale turns its
    logits around.  Lengths on and off the tile edges."""
    c = Made(tr, np.random.default_rng(50 + G), "e4m3", 16, [17, 33, 100, 64, 0, 1, 700], 6, d)
    c.ks.copy_(torch.tensor([0.0, -0.02, 0.015, 1e-42, -0.0, -0.5]))
    if reach:
        widened(tr, c, reach)
    Q = c.queries(6 * G, 4.0)
    before = c.scores.clone()
    O, lse = c.attend(Q, d ** -0.5, accumulate=True)
    c.check(Q, d ** -0.5, O, lse, before)
    n = 33
    flat = torch.tensor(float(np.log(n)), device="cuda")
    assert torch.allclose(lse[1, :G], flat) and torch.allclose(lse[1, 3 * G:5 * G], flat)


@pytest.mark.parametrize("reach", [0, 1 << 18])
@pytest.mark.parametrize("factor", [2.0 ** -133, 2.0 ** -127, 2.0 ** -120, 1e-30, 2.0 ** 60])
def test_decode_e4m3_tiny_queries(tr, reach, factor):
    """Queries so small that every weight is the same, under an ordinary scale (what they are multiplied with inside
    goes below the smallest number), and large ones with a tiny scale of the head."""
    c = Made(tr, np.random.default_rng(51), "e4m3", 16, [17, 33, 100], 2, 128)
    c.ks.copy_(torch.tensor([0.01, 1e-10]) if factor < 1 else torch.tensor([2.0 ** -60, -2.0 ** -130]))
    if reach:
        widened(tr, c, reach)
    Q = c.queries(8, 1.0).float().sign().mul(factor).to(c.cache.row_dtype)
    Q[:, 1] = 0.0
    assert Q[:, 0].float().abs().min() > 0
    before = c.scores.clone()
    O, lse = c.attend(Q, 0.088, accumulate=True)
    c.check(Q, 0.088, O, lse, before)


@pytest.mark.parametrize("reach", [0, 1 << 14, 1 << 18])
@pytest.mark.parametrize("G", [4, 12])
@pytest.mark.parametrize("q2,k2,scale2", [(66, 62, -126), (98, 28, -125), (126, 0, -125), (-126, 120, 5),
                                          (10, 116, -125), (-8, 126, -119), (0, 126, -126),
                                          (70, 62, -131), (90, 60, -145)])
def test_decode_products_beyond_fp32(tr, reach, G, q2, k2, scale2):
    """bf16 rows whose products with the queries pass fp32's range, or come near it, while the scaled logits are
    ordinary ones."""
    c = Made(tr, np.random.default_rng(52), "bf16", 16, [17, 40, 300], 2, 128)
    for b in range(3):
        c.rows_k[b] = (c.rows_k[b].double() * 2.0 ** k2).clamp(-3e38, 3e38).bfloat16()
        c.put(c.K, b, c.rows_k[b])
    if reach:
        widened(tr, c, reach)
    Q = (c.queries(2 * G, 1.0).double() * 2.0 ** q2).clamp(-3e38, 3e38).bfloat16()
    scale = 1.5 * 2.0 ** scale2
    before = c.scores.clone()
    O, lse = c.attend(Q, scale, accumulate=True)
    c.check(Q, scale, O, lse, before)


def test_decode_repeats_bit_for_bit_and_shares_pages(tr):
    """Equal calls give equal bits, alone and on two streams at once with a workspace each; sequences may share pages."""
    c = Made(tr, np.random.default_rng(9), "bf16", 16, [3000, 3000, 100, 0], 2, 128)
    c.pt_host[1, :100] = c.pt_host[0, :100]  # a common prompt
    c.pt.copy_(c.pt_host)
    c.rows_k[1][:, :1600], c.rows_v[1][:, :1600] = c.rows_k[0][:, :1600], c.rows_v[0][:, :1600]
    Q = c.queries(8, 2.0)
    s0 = c.scores.clone()
    O, lse = c.attend(Q, 0.09, accumulate=True)
    c.check(Q, 0.09, O, lse, s0)
    s1 = c.scores.clone()
    for _ in range(3):
        c.scores.copy_(s0)
        O2, lse2 = c.attend(Q, 0.09, accumulate=True)
        assert torch.equal(O, O2) and torch.equal(lse, lse2) and torch.equal(c.scores, s1)
    Qd = Q.cuda()
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for st in streams:
        with torch.cuda.stream(st):
            for _ in range(10):
                outs.append(c.attend(Qd, 0.09)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(O, o) for o in outs)


def test_decode_graph_follows_lengths_pages_and_inputs(tr):
    """One captured call, replayed with other lengths (down to 0), another page table and other queries."""
    rng = np.random.default_rng(10)
    c = Made(tr, rng, "bf16", 16, [900, 40, 2000], 2, 128)
    Q = c.queries(8, 2.0).cuda()
    O, lse = torch.empty(3, 8, 128, device="cuda"), torch.empty(3, 8, device="cuda")
    ws = tr.workspace(tr.tr_decode_attn_workspace_bytes(c.cache, 8, True))
    call = lambda: tr.tr_decode_attn(Q, c.cache, O, 0.09, ws, lse=lse, accumulate=True)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    full_k, full_v = c.rows_k, c.rows_v
    for lengths, order in (([900, 40, 2000], [0, 1, 2]), ([0, 17, 5], [0, 1, 2]), ([900, 2000, 33], [0, 2, 1])):
        Q.copy_(c.queries(8, 2.0))
        c.pt.copy_(c.pt_host[order])
        c.L.copy_(torch.tensor(lengths, dtype=torch.int32))
        c.lengths = lengths
        c.rows_k = [full_k[o][:, :n] for o, n in zip(order, lengths)]
        c.rows_v = [full_v[o][:, :n] for o, n in zip(order, lengths)]
        before = c.scores.clone()
        O.fill_(float("nan"))
        graph.replay()
        c.check(Q, 0.09, O, lse, before)


def test_decode_bad_lengths_and_pages_are_reported(tr):
    """The host's and the kernels' own checks turn each into a status bit; the other sequences are right."""
    c = Made(tr, np.random.default_rng(11), "bf16", 16, [50, 60, 70, 80], 2, 128)
    Q = c.queries(4)
    c.L.copy_(torch.tensor([50, -1, 70, c.cap + 1], dtype=torch.int32))
    before = c.scores.clone()
    O, lse = c.attend(Q, 0.1, accumulate=True)
    assert tr.tr_get_status() == tr.TR_DEV_BAD_LENGTH
    keep, c.lengths = c.lengths, [50, 0, 70, 0]
    for b in (1, 3):
        c.rows_k[b], c.rows_v[b] = c.rows_k[b][:, :0], c.rows_v[b][:, :0]
    c.check(Q, 0.1, O, lse, before)
    for bad in (-1, c.K.shape[0], 1 << 30):
        c2 = Made(tr, np.random.default_rng(12), "bf16", 16, [50, 60, 70], 2, 128)
        c2.pt[1, 2] = bad
        O, lse = c2.attend(c2.queries(4), 0.1, accumulate=True)
        assert tr.tr_get_status() == tr.TR_DEV_BAD_PAGE
    c3 = Made(tr, np.random.default_rng(13), "bf16", 16, [50, 60, 70], 2, 128)
    Q = c3.queries(4)
    c3.pt[1, 2] = -5
    O, lse = c3.attend(Q, 0.1)
    assert tr.tr_get_status() == tr.TR_DEV_BAD_PAGE
    sub = [0, 2]
    c3.lengths = [50, 70]
    c3.rows_k, c3.rows_v = [c3.rows_k[b] for b in sub], [c3.rows_v[b] for b in sub]
    c3.check(Q[sub], 0.1, O[sub], lse[sub])


def test_offsets_past_32_bits(tr):
    """A pool of more than 2^32 bytes per tensor whose used pages lie at its end, appended to, attended and cut."""
    P, ps, Hkv, d = 300_000, 16, 8, 128  # 4.9e9 elements
    K = torch.empty(P, Hkv, ps, d, dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    pt = torch.tensor([[P - 1, P - 3, P - 2, 5]], dtype=torch.int32, device="cuda")
    L = torch.zeros(1, dtype=torch.int32, device="cuda")
    scores = torch.empty(1, Hkv, 64, device="cuda")
    cache = tr.KVCache(K, V, L, page_table=pt, scores=scores)
    g = torch.Generator().manual_seed(4)
    new = [torch.randn(1, 60, Hkv, d, generator=g).bfloat16() for _ in range(2)]
    tr.tr_kv_append(new[0].cuda(), new[1].cuda(), cache, tr.workspace(tr.tr_kv_append_workspace_bytes(cache)))
    assert torch.equal(K[P - 3, 5].cpu(), new[0][0, 16:32, 5])
    Q = torch.randn(1, 16, d, generator=g).bfloat16()

    def attend(rows):
        O = torch.empty(1, 16, d, device="cuda")
        tr.tr_decode_attn(Q.cuda(), cache, O, 0.1,
                          tr.workspace(tr.tr_decode_attn_workspace_bytes(cache, 16, True)), accumulate=True)
        for h in range(Hkv):
            k, v = (x[0, rows[h], h].double().numpy()[None] for x in new)
            ref, _, _ = oracle.decode_attention(Q[0, 2 * h:2 * h + 2].double().numpy(), k, v, 0.1)
            assert np.abs(O[0, 2 * h:2 * h + 2].cpu().double().numpy() - ref).max() < 1e-4
    attend([list(range(60))] * Hkv)
    keep = [oracle.evict_keep(scores[0, h, :60].cpu().numpy(), 35, 9) for h in range(Hkv)]
    tr.tr_kv_evict(cache, 35, 9, tr.workspace(tr.tr_kv_evict_workspace_bytes(cache, 35)))
    assert L.item() == 35
    attend(keep)


@pytest.mark.parametrize("n", [0, 1])
def test_decode_most_query_heads(tr, n):
    """The most query heads that the call takes (groups of 65793): O's elements come within 128 of 2^31."""
    Hkv, Hq, d = 255, (1 << 24) - 1, 128
    K = torch.randn(1, Hkv, 16, d, device="cuda").bfloat16()
    V = torch.randn(1, Hkv, 16, d, device="cuda").bfloat16()
    cache = tr.KVCache(K, V, torch.tensor([n], dtype=torch.int32, device="cuda"))
    Q = torch.zeros(1, Hq, d, dtype=torch.bfloat16, device="cuda")
    O = torch.full((1, Hq, d), float("nan"), device="cuda")
    lse = torch.full((1, Hq), float("nan"), device="cuda")
    ws = torch.empty(tr.tr_decode_attn_workspace_bytes(cache, Hq), dtype=torch.uint8, device="cuda")
    tr.tr_decode_attn(Q, cache, O, d ** -0.5, ws, lse)
    # one row has the weight 1, logits of 0 a logarithm of 0
    want = V[0, :, :1].float() * n
    assert bool((O.view(Hkv, Hq // Hkv, d) == want).all())
    assert bool((lse == (0.0 if n else -float("inf"))).all())


def test_tensors_of_the_binding(tr):
    """What the Python layer refuses beyond the host checks of the library."""
    K = torch.zeros(2, 4, 64, 128, dtype=torch.bfloat16, device="cuda")
    L = torch.zeros(2, dtype=torch.int32, device="cuda")
    sc = torch.zeros(2, 4, 64, device="cuda")
    pt = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    ks = torch.ones(4, device="cuda")
    bad = [dict(V=K.half()), dict(V=K[:1]), dict(V=K.transpose(1, 2).contiguous().transpose(1, 2)), dict(L=L.long()),
           dict(L=L[:1]), dict(L=L.view(2, 1)), dict(page_table=pt.long()), dict(page_table=pt[:1]),
           dict(page_table=pt[0]), dict(scores=sc.double()), dict(scores=sc[:, :, :63]), dict(scores=sc[:, :3]),
           dict(k_scale=ks), dict(k_scale=ks, v_scale=ks), dict(L=L.cpu()), dict(scores=sc.cpu()),
           dict(K=K[..., ::2], V=K[..., ::2]), dict(scores=sc.transpose(1, 2))]
    for kw in bad:
        with pytest.raises(ValueError):
            tr.KVCache(**{**dict(K=K, V=K, L=L), **kw})
    K8 = K.to(torch.float8_e4m3fn)
    for kw in (dict(), dict(k_scale=ks), dict(k_scale=ks, v_scale=ks[:3]), dict(k_scale=ks, v_scale=ks.double())):
        with pytest.raises(ValueError):
            tr.KVCache(K8, K8, L, **kw)
    c = tr.KVCache(K, K.clone(), L, scores=sc)
    ws = tr.workspace(1 << 20)
    Q = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    O = torch.zeros(2, 8, 128, device="cuda")
    lse = torch.zeros(2, 8, device="cuda")
    for kw in (dict(Q=Q.half()), dict(Q=Q[:1]), dict(Q=Q[:, :, :64]), dict(Q=Q[:, ::2]), dict(O=O.half()),
               dict(O=O[:, :4]), dict(lse=lse[:, :4]), dict(lse=lse.double()), dict(ws=O), dict(Q=Q.cpu())):
        with pytest.raises(ValueError):
            tr.tr_decode_attn(**{**dict(Q=Q, cache=c, O=O, scale=0.1, ws=ws, lse=lse), **kw})
    with pytest.raises(tr.TRError):
        tr.tr_decode_attn(Q, c, O, 0.0, ws)
    with pytest.raises(tr.TRError):
        tr.tr_decode_attn(Q, c, O, 0.1, ws[:64], accumulate=True)
    n = torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16, device="cuda")
    cnt = torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw in (dict(Kn=n.half(), Vn=n.half()), dict(Kn=n[:1]), dict(Vn=n[:, :2]), dict(count=cnt.long()),
               dict(count=cnt[:1]), dict(Kn=n[:, :, :2]), dict(Kn=n.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            tr.tr_kv_append(**{**dict(Kn=n, Vn=n, cache=c, ws=ws, count=cnt), **kw})
    for budget, recent in ((1 << 32, 0), ((1 << 32) + 8, 2), (-3, 0), (8, (1 << 32) + 1)):
        with pytest.raises(ValueError):
            tr.tr_kv_evict(c, budget, recent, ws)
    with pytest.raises(tr.TRError):
        tr.tr_kv_evict(c, 8, 9, ws)
    with pytest.raises(tr.TRError):
        tr.tr_kv_evict(tr.KVCache(K, K.clone(), L), 8, 2, ws)


# ----------------------------------------------------------------------------
# appending
# ----------------------------------------------------------------------------

def check_append(c, T, count):
    """tr_kv_append's rows, scores and lengths against the definition; all else is left as it was."""
    B, Hkv, d = len(c.lengths), c.Hkv, c.d
    wide = c.cache.row_dtype
    new = [(torch.randn(B, T, Hkv, d, generator=c.g) * (3.0 if c.type == "e4m3" else 1.0)).to(wide) for _ in range(2)]
    if c.type == "e4m3":  # clamped values, the smallest ones, ties and NaN
        new[0][0, 0, 0, :6] = torch.tensor([1e9, -1e9, 1e-9, float("nan"), float("inf"), -float("inf")])
        s = float(c.ks[0])
        new[1][0, 0, 0, :4] = torch.tensor([2.0625 * s, 2.1875 * s, 2 ** -10 * s, 3 * 2 ** -10 * s])
    old = [raw(c.K).clone(), raw(c.V).clone(), c.scores.clone()]
    cnt = None if count is None else torch.tensor(count, dtype=torch.int32, device="cuda")
    ws = torch.full((c.tr.tr_kv_append_workspace_bytes(c.cache),), 0xA5, dtype=torch.uint8, device="cuda")
    c.tr.tr_kv_append(new[0].cuda(), new[1].cuda(), c.cache, ws, count=cnt)
    count = [T] * B if count is None else count
    want = [raw(c.K).clone(), raw(c.V).clone(), c.scores.clone()]
    for w, o in zip(want, old):
        w.copy_(o)
    for b, (n, t) in enumerate(zip(c.lengths, count)):
        for x, w, rows, scale in ((new[0], want[0], c.rows_k, c.ks), (new[1], want[1], c.rows_v, c.vs)):
            r = x[b, :t].transpose(0, 1)
            if scale is not None:  # fp32 division, then one rounding
                q = oracle.e4m3_round((r.float() / scale.cpu()[:, None, None]).numpy())
                r = torch.from_numpy(q).float().to(TYPES["e4m3"])
            rows[b] = raw(torch.cat([raw(rows[b]), raw(r.contiguous())], 1).view(TYPES[c.type])).view(TYPES[c.type])
            for i in range(t):
                p = n + i
                at = (b, p) if c.pt is None else (int(c.pt_host[b, p // c.ps]), p % c.ps)
                w[at[0], :, at[1]] = raw(r[:, i].contiguous()).cuda()
        want[2][b, :, n:n + t] = 0
    if c.type == "e4m3":  # NaN has two codes
        f8 = TYPES["e4m3"]
        for got, w in ((c.K, want[0]), (c.V, want[1])):
            assert torch.equal(torch.nan_to_num(got.float(), 1e6), torch.nan_to_num(w.view(f8).float(), 1e6))
    else:
        assert torch.equal(raw(c.K), want[0]) and torch.equal(raw(c.V), want[1])
    assert torch.equal(c.scores, want[2])
    c.lengths = [n + t for n, t in zip(c.lengths, count)]
    assert c.L.tolist() == c.lengths


@pytest.mark.parametrize("type", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["dense", "dense_nhd", "wide", 1, 16, 64, "nhd16"])
def test_append(tr, type, d, layout):
    c = Made(tr, np.random.default_rng(20), type, layout, [0, 5, 16, 31, 100], 3, d, extra=60)
    check_append(c, 1, None)
    check_append(c, 37, [37, 0, 1, 16, 36])
    check_append(c, 2, [0, 0, 0, 0, 0])
    check_append(c, 4, None)


@pytest.mark.parametrize("Hkv", [256, 257, 300])
def test_append_many_heads_e4m3(tr, Hkv):
    """Up to 256 heads' scales are kept by a CTA, of more each thread takes its own."""
    c = Made(tr, np.random.default_rng(56), "e4m3", 16, [5, 0, 17], Hkv, 64, extra=20)
    check_append(c, 1, None)
    check_append(c, 9, [9, 3, 0])


def test_append_and_evict_most_sequences(tr):
    c = Made(tr, np.random.default_rng(57), "bf16", 16, [(7 * b) % 40 for b in range(1024)], 1, 64, extra=8)
    check_append(c, 3, [b % 4 for b in range(1024)])
    check_evict(c, 11, 3)


def test_append_exactly_full_and_over(tr):
    """Rows up to the last place; one more is refused for that sequence alone."""
    c = Made(tr, np.random.default_rng(21), "bf16", "dense", [60, 50, 64], 2, 128)
    assert c.cap == 64
    check_append(c, 4, [4, 4, 0])
    old = [raw(c.K).clone(), raw(c.V).clone(), c.scores.clone()]
    n = torch.randn(3, 11, 2, 128).bfloat16().cuda()
    ws = tr.workspace(tr.tr_kv_append_workspace_bytes(c.cache))
    tr.tr_kv_append(n, n, c.cache, ws, count=torch.tensor([1, 11, 1], dtype=torch.int32, device="cuda"))
    assert tr.tr_get_status() == tr.TR_DEV_CACHE_FULL
    assert c.L.tolist() == [64, 54, 64]
    for x, o in zip((raw(c.K), raw(c.V), c.scores), old):
        assert torch.equal(x, o)


@pytest.mark.parametrize("T", [3, 200])
def test_append_bad_inputs_are_reported(tr, T):
    c = Made(tr, np.random.default_rng(22), "bf16", 16, [20, 20, 20, 20], 4, 128, extra=200)
    n = torch.randn(4, T, 4, 128).bfloat16().cuda()
    ws = tr.workspace(tr.tr_kv_append_workspace_bytes(c.cache))
    old = raw(c.K).clone()
    for cnt, L, bit in (([T + 1, -1, 0, 0], [20] * 4, tr.TR_DEV_BAD_LENGTH),
                        ([1, 1, 0, 0], [-1, c.cap + 1, 20, 20], tr.TR_DEV_BAD_LENGTH)):
        c.L.copy_(torch.tensor(L, dtype=torch.int32))
        tr.tr_kv_append(n, n, c.cache, ws, count=torch.tensor(cnt, dtype=torch.int32, device="cuda"))
        assert tr.tr_get_status() == bit
        assert c.L.tolist() == L and torch.equal(raw(c.K), old)
    c.L.fill_(20)
    c.pt[1, 1] = -1      # the page that row 20 goes to
    c.pt[2, 0] = -1      # a page that no new row needs
    tr.tr_kv_append(n, n, c.cache, ws)
    assert tr.tr_get_status() == tr.TR_DEV_BAD_PAGE
    assert c.L.tolist() == [20 + T, 20, 20 + T, 20 + T]


def test_append_into_graph(tr):
    """A captured append goes on where the last replay ended."""
    c = Made(tr, np.random.default_rng(23), "bf16", 16, [3, 0], 2, 128, extra=40)
    n = torch.randn(2, 5, 2, 128).bfloat16().cuda()
    ws = tr.workspace(tr.tr_kv_append_workspace_bytes(c.cache))
    L0 = c.L.clone()
    tr.tr_kv_append(n, n, c.cache, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tr.tr_kv_append(n, n, c.cache, ws)
    c.L.copy_(L0)
    rows = []
    for _ in range(4):
        n.copy_(torch.randn(2, 5, 2, 128))
        rows.append(n.cpu())
        graph.replay()
    assert c.L.tolist() == [23, 20]
    for b, n0 in ((0, 3), (1, 0)):
        assert torch.equal(c.get(c.K, b, n0 + 20)[:, n0:], torch.cat([r[b] for r in rows]).transpose(0, 1))


# ----------------------------------------------------------------------------
# eviction
# ----------------------------------------------------------------------------

def check_evict(c, budget, recent):
    B = len(c.lengths)
    old_sc = c.scores.clone()
    old = [[c.get(x, b, n) for b, n in enumerate(c.lengths)] for x in (c.K, c.V)]
    pools = [raw(c.K).clone(), raw(c.V).clone()]
    ws = torch.full((c.tr.tr_kv_evict_workspace_bytes(c.cache, budget),), 0xA5, dtype=torch.uint8, device="cuda")
    c.tr.tr_kv_evict(c.cache, budget, recent, ws)
    for b, n in enumerate(c.lengths):
        m = min(n, budget)
        sc = old_sc[b].cpu()
        keep = [oracle.evict_keep(sc[h, :n].numpy(), budget, recent) for h in range(c.Hkv)]
        for x, o, rows in ((c.K, old[0], c.rows_k), (c.V, old[1], c.rows_v)):
            got, was = c.get(x, b, n), o[b]
            want = torch.cat([torch.stack([raw(was)[h, keep[h]] for h in range(c.Hkv)]), raw(was)[:, m:]], 1)
            assert torch.equal(raw(got), want), "rows of sequence %d" % b
            rows[b] = got[:, :m].contiguous()
        want = sc.clone()
        for h in range(c.Hkv):
            want[h, :m] = sc[h, keep[h]]
        assert torch.equal(c.scores[b].cpu().view(torch.int32), want.view(torch.int32)), "scores of sequence %d" % b
    # nothing outside the sequences' rows is written
    for x, o in zip((c.K, c.V), pools):
        mask = torch.ones(x.shape[0], x.shape[2], dtype=torch.bool)
        for b, n in enumerate(c.lengths):
            for p in range(min(n, budget)):
                at = (b, p) if c.pt is None else (int(c.pt_host[b, p // c.ps]), p % c.ps)
                mask[at] = False
        keepers = mask.cuda()
        assert torch.equal(raw(x).transpose(1, 2)[keepers], o.transpose(1, 2)[keepers])
    c.lengths = [min(n, budget) for n in c.lengths]
    assert c.L.tolist() == c.lengths


@pytest.mark.parametrize("type,d", [("bf16", 128), ("f16", 64), ("e4m3", 128), ("e4m3", 64)])
@pytest.mark.parametrize("layout", ["dense", "dense_nhd", "wide", 1, 16, "nhd64"])
@pytest.mark.parametrize("budget,recent", [(40, 8), (65, 0), (17, 17), (1, 0), (1, 1), (500, 3)])
def test_evict(tr, type, d, layout, budget, recent):
    c = Made(tr, np.random.default_rng(30), type, layout, [0, 1, budget, budget + 1, 130, 41, 300, 64], 2, d)
    check_evict(c, budget, recent)
    if budget > 20:
        check_evict(c, budget // 2, min(recent, 3))   # a second time on what is left


@pytest.mark.parametrize("n,budget,recent", [(1025, 600, 100), (5000, 1024, 256), (5000, 4999, 0), (20000, 9000, 1),
                                             (2050, 2048, 2047), (40000, 33, 1), (4096, 1, 0)])
def test_evict_long(tr, n, budget, recent):
    c = Made(tr, np.random.default_rng(31), "bf16", 64, [n, n // 2 + 1], 2, 64)
    check_evict(c, budget, recent)


@pytest.mark.parametrize("type,d,layout", [("bf16", 128, "dense"), ("e4m3", 64, 16), ("f16", 64, "nhd64")])
@pytest.mark.parametrize("budget,recent", [(300, 40), (64, 64), (900, 0)])
def test_evict_many_pairs(tr, type, d, layout, budget, recent):
    """More (sequence, head) pairs than SMs: whole rows by one CTA each."""
    c = Made(tr, np.random.default_rng(36), type, layout, [37 * b % 1200 for b in range(44)], 4, d)
    check_evict(c, budget, recent)


@pytest.mark.parametrize("type,d,n,budget", [("bf16", 128, 6000, 4700), ("bf16", 128, 20000, 4700),
                                             ("f16", 64, 14000, 4700), ("e4m3", 128, 6000, 4700),
                                             ("e4m3", 64, 19000, 8000)])
@pytest.mark.parametrize("layout", ["wide", 1, 16, "nhd64"])
@pytest.mark.parametrize("recent", [0, 700, 4700])
def test_evict_few_pairs_of_many_rows(tr, type, d, n, budget, layout, recent):
    """Few pairs that keep many rows: those from behind the budget move apart, in two stretches, after the others."""
    c = Made(tr, np.random.default_rng(38), type, layout, [n, budget + 1], 2, d)
    check_evict(c, budget, recent)


@pytest.mark.parametrize("budget,recent", [(2000, 10), (6000, 5000), (7900, 100), (4096, 0), (8191, 0)])
def test_evict_around_the_halfway_mark(tr, budget, recent):
    """Few pairs: rows from behind the budget move apart from the others, whatever part of the kept ones they are."""
    c = Made(tr, np.random.default_rng(37), "bf16", "dense", [8192, 4097, 8000], 2, 64)
    check_evict(c, budget, recent)


@pytest.mark.parametrize("n,budget,recent", [(400_000, 150_000, 1000), (330_000, 329_999, 5), (70_000, 1, 0)])
def test_evict_very_long(tr, n, budget, recent):
    """More rows than the shared memory of a whole cluster holds scores of (8 x 40960), and up to that many."""
    c = Made(tr, np.random.default_rng(35), "e4m3", 256, [n], 1, 64)
    c.scores.copy_((c.scores * 500).round() / 500)   # ties
    check_evict(c, budget, recent)


@pytest.mark.parametrize("n", [131071, 131072, 131073, 131105])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_where_a_cluster_stops_holding_the_scores(tr, n, ties):
    """One pair, a cluster of eight CTAs: 16384 scores of each are held in its registers, of more they are read again."""
    c = Made(tr, np.random.default_rng(53), "e4m3", 256, [n], 1, 64)
    if ties:
        c.scores.copy_((c.scores * 50).round() / 50)
    check_evict(c, 40_000, 0)


@pytest.mark.parametrize("n", [16384, 16385, 20011])
def test_evict_many_pairs_of_long_sequences(tr, n):
    """So many pairs that one CTA chooses the rows of each, of which it holds 16384: more are read again in every pass."""
    lengths = [0, n + 37, 3, 700, n] + [0] * 35
    c = Made(tr, np.random.default_rng(54), "e4m3", 64, lengths, 8, 64)
    c.scores.copy_((c.scores * 200).round() / 200)
    check_evict(c, 600, 37)


@pytest.mark.parametrize("scale", [1.0, 0.0123, 1e-3, 3e-19, 1e-25, 7e18, 2e30])
def test_append_divides_exactly(tr, scale):
    """Every quotient that decides between two 8-bit values: the rows lie on and next to the rounding borders."""
    T, d = 64, 128
    K = torch.zeros(1, 1, 128, d, device="cuda").to(TYPES["e4m3"])
    V, L = K.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    ks = torch.tensor([scale], device="cuda")
    cache = tr.KVCache(K, V, L, k_scale=ks, v_scale=ks * 1.7)
    grid = torch.arange(127, dtype=torch.uint8).view(TYPES["e4m3"]).double()
    grid = torch.cat([grid, torch.tensor([480.0, 1000.0, 1025.0, 1e6], dtype=torch.float64)])
    mid = (grid[1:] + grid[:-1]) / 2
    x = torch.cat([grid, mid, -mid]) * float(ks)                  # borders, as near as bf16 comes
    x = x.bfloat16().view(torch.int16)
    x = torch.cat([x, x + 1, x - 1, x + 2]).view(torch.bfloat16)
    rng = torch.Generator().manual_seed(1)
    more = torch.randn(T * d - len(x), generator=rng, dtype=torch.float64) * 10 ** (torch.rand(T * d - len(x), generator=rng) * 6 - 3)
    x = torch.cat([x, (more * float(ks)).bfloat16()]).view(1, T, 1, d)
    tr.tr_kv_append(x.cuda(), x.cuda(), cache, tr.workspace(tr.tr_kv_append_workspace_bytes(cache)))
    for got, s in ((K, ks), (V, ks * 1.7)):
        want = oracle.e4m3_round((x[0, :, 0].float() / s.cpu()).numpy())
        assert np.array_equal(got[0, 0, :T].double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("scale", [1.0, 0.0123, 2.0 ** -59, 2.0 ** 59, 3e-19, 1e-25, 2e30, -0.5])
def test_append_keeps_the_sign_of_zero(tr, scale):
    """-0, and what is too small to be held, keep their signs: bytes as the division and one rounding give them, with
    scales of both ways that the division is done."""
    d, T = 64, 8
    K = torch.zeros(1, 1, 16, d, device="cuda").to(TYPES["e4m3"])
    V, L = K.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.tensor([scale], device="cuda")
    cache = tr.KVCache(K, V, L, k_scale=s, v_scale=s)
    x = torch.tensor([0.0, -0.0, 1e-20, -1e-20, 2.0 ** -133, -2.0 ** -133, 1e-38, -1e-38], dtype=torch.float64)
    y = torch.tensor([1.0, -1.0, 2.0 ** -11, -2.0 ** -11, 2.0 ** -10, -2.0 ** -10, 2.0 ** -9, -2.0 ** -9, 448.0, -448.0,
                      1e6, -1e6], dtype=torch.float64) * abs(scale)
    x = torch.cat([x, y, -x, -y])
    x = torch.cat([x] * 13)[:T * d].bfloat16().view(1, T, 1, d)
    tr.tr_kv_append(x.cuda(), (-x).cuda(), cache, tr.workspace(tr.tr_kv_append_workspace_bytes(cache)))
    for got, rows in ((K, x), (V, -x)):
        q = oracle.e4m3_round((rows[0, :, 0].float() / s.cpu()).numpy())
        want = torch.from_numpy(q).float().to(TYPES["e4m3"])
        assert torch.equal(raw(got[0, 0, :T]).cpu(), raw(want))


@pytest.mark.parametrize("kind", ["equal", "zeros", "few", "special", "negative", "sorted", "reversed", "tiny"])
def test_evict_ties_and_special_scores(tr, kind):
    """Ties go to the lower position; NaN ranks below -inf; -0 equals +0; order is that of the values."""
    rng = np.random.default_rng(32)
    c = Made(tr, rng, "bf16", 16, [300, 77, 1100], 3, 64)
    s = rng.normal(size=c.scores.shape).astype(np.float32)
    if kind == "equal":
        s[:] = 0.25
    elif kind == "zeros":
        s = np.where(rng.random(s.shape) < 0.5, np.float32(0.0), np.float32(-0.0))
    elif kind == "few":
        s = rng.integers(0, 3, s.shape).astype(np.float32)
    elif kind == "special":
        s = rng.choice(np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, 3e38, 1e-45, -1e-45], np.float32), s.shape)
    elif kind == "negative":
        s = -np.abs(s)
    elif kind == "sorted":
        s = np.sort(s, axis=2)
    elif kind == "reversed":
        s = np.ascontiguousarray(np.sort(s, axis=2)[:, :, ::-1])
    else:
        s = (s * 1e-40).astype(np.float32)
    c.scores.copy_(torch.from_numpy(s))
    check_evict(c, 64, 10)


def test_evict_bad_lengths_and_pages_leave_the_sequence(tr):
    c = Made(tr, np.random.default_rng(33), "bf16", 16, [100, 100, 100, 100], 2, 64)
    c.L.copy_(torch.tensor([100, -1, c.cap + 1, 100], dtype=torch.int32))
    c.pt[3, 6] = 1 << 20
    K0, s0 = raw(c.K).clone(), c.scores.clone()
    tr.tr_kv_evict(c.cache, 50, 10, tr.workspace(tr.tr_kv_evict_workspace_bytes(c.cache, 50)))
    assert tr.tr_get_status() == tr.TR_DEV_BAD_LENGTH | tr.TR_DEV_BAD_PAGE
    assert c.L.tolist() == [50, -1, c.cap + 1, 100]
    for b in (1, 2, 3):
        used = c.pt_host[b, :7].long().cuda()
        assert torch.equal(raw(c.K)[used], K0[used]) and torch.equal(c.scores[b], s0[b])
    # a budget beyond the cache: nothing to do, lengths are still looked at
    tr.tr_kv_evict(c.cache, 1 << 30, 0, tr.workspace(tr.tr_kv_evict_workspace_bytes(c.cache, 1 << 30)))
    assert tr.tr_get_status() == tr.TR_DEV_BAD_LENGTH
    assert c.L.tolist() == [50, -1, c.cap + 1, 100]


def test_evict_in_a_graph(tr):
    """One captured eviction, replayed on lengths over and within the budget."""
    c = Made(tr, np.random.default_rng(34), "bf16", 16, [200, 90, 150], 2, 64)
    ws = tr.workspace(tr.tr_kv_evict_workspace_bytes(c.cache, 80))
    L0 = c.L.clone()
    c.L.zero_()
    tr.tr_kv_evict(c.cache, 80, 16, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tr.tr_kv_evict(c.cache, 80, 16, ws)
    for lengths in (L0.tolist(), [200, 60, 81]):
        c.L.copy_(torch.tensor(lengths, dtype=torch.int32))
        sc, K = c.scores.clone(), [c.get(c.K, b, n) for b, n in enumerate(lengths)]
        graph.replay()
        assert c.L.tolist() == [min(n, 80) for n in lengths]
        for b, n in enumerate(lengths):
            for h in range(2):
                keep = oracle.evict_keep(sc[b, h, :n].cpu().numpy(), 80, 16)
                assert torch.equal(c.get(c.K, b, len(keep))[h], K[b][h, keep])


# ----------------------------------------------------------------------------
# together
# ----------------------------------------------------------------------------

FIRST_CALLS = """
import torch, free_speculative_decoding_gb300 as tr
B, H, cap, d = 2, 3, 9000, 64
K = torch.randn(B, H, cap, d, device="cuda").bfloat16()
V, sc = K.clone(), torch.rand(B, H, cap, device="cuda")
L0 = torch.tensor([8000, 77], dtype=torch.int32, device="cuda")
L = L0.clone()
c = tr.KVCache(K, V, L, scores=sc)
Q, O = torch.randn(B, 6, d, device="cuda").bfloat16(), torch.zeros(B, 6, d, device="cuda")
n = torch.randn(B, 500, H, d, device="cuda").bfloat16()
ws = [tr.workspace(x) for x in (tr.tr_kv_append_workspace_bytes(c), tr.tr_decode_attn_workspace_bytes(c, 6, True),
                                tr.tr_kv_evict_workspace_bytes(c, 300))]
def step():
    tr.tr_kv_append(n, n, c, ws[0])
    tr.tr_decode_attn(Q, c, O, 0.125, ws[1], accumulate=True)
    tr.tr_kv_evict(c, 300, 40, ws[2])
K0, V0, s0 = K.clone(), V.clone(), sc.clone()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
got = [x.clone() for x in (O, K, V, sc, L)]
for x, y in ((K, K0), (V, V0), (sc, s0), (L, L0)):
    x.copy_(y)
O.zero_()
step()
assert all(torch.equal(x, y) for x, y in zip(got, (O, K, V, sc, L)))
assert L.tolist() == [300, 300] and tr.tr_get_status() == 0
print("fine")
"""


def test_first_calls_of_a_process_inside_a_capture(tr):
    """Nothing has to run before a capture: all three calls are captured as a process's first, and replay to what
    they do eagerly."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def test_calls_behind_a_join_of_two_streams(tr):
    """Inputs made on a second stream and joined by an event right before each call, eagerly and in a capture (where
    each call's first kernel then has two predecessors), two graphs of the same operators among them."""
    c = Made(tr, np.random.default_rng(42), "bf16", 16, [700, 30, 1500], 2, 128, extra=400)
    a, o = tr.workspace(tr.tr_kv_append_workspace_bytes(c.cache)), tr.workspace(
        tr.tr_decode_attn_workspace_bytes(c.cache, 8, True))
    e = tr.workspace(tr.tr_kv_evict_workspace_bytes(c.cache, 500))
    src = [torch.randn(3, 70, 2, 128, generator=c.g).bfloat16().cuda(), c.queries(8, 2.0).cuda()]
    n, Q = torch.zeros_like(src[0]), torch.zeros_like(src[1])
    O = torch.zeros(3, 8, 128, device="cuda")
    busy = torch.randn(4 << 20, device="cuda")
    side = torch.cuda.Stream()

    def both(f):
        """f on the side stream while this one works; then joined."""
        now = torch.cuda.current_stream()
        side.wait_stream(now)
        with torch.cuda.stream(side):
            torch.sin(busy)
            f()
        torch.cos(busy)
        now.wait_stream(side)

    def step():
        both(lambda: n.copy_(src[0] * 2))
        tr.tr_kv_append(n, n, c.cache, a)
        both(lambda: Q.copy_(src[1] * 0.5))
        tr.tr_decode_attn(Q, c.cache, O, 0.09, o, accumulate=True)
        both(lambda: torch.cos(busy))
        tr.tr_kv_evict(c.cache, 500, 60, e)

    state = [raw(c.K), raw(c.V), c.scores, c.L]
    start = [x.clone() for x in state]
    outs = []
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for way in (None, 0, 1, 0):
        for x, y in zip(state, start):
            x.copy_(y)
        n.zero_(), Q.zero_(), O.zero_()
        torch.cuda.synchronize()
        if way is None:
            step()
        else:
            if not outs[way + 1:]:
                with torch.cuda.graph(graphs[way]):
                    step()
            graphs[way].replay()
        torch.cuda.synchronize()
        outs.append([O.clone()] + [x.clone() for x in state])
    for got in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(outs[0], got))
    assert c.L.tolist() == [500, 100, 500]


@pytest.mark.parametrize("layout", ["dense", 16])
def test_back_to_back_calls_see_each_other(tr, layout):
    """Append, attention and eviction queued without a pause between them (each may be set up while the one before it
    ends) read what the one before wrote: the same as with a synchronisation after every call."""
    outs = []
    for wait in (False, True):
        c = Made(tr, np.random.default_rng(41), "bf16", layout, [700, 3, 0, 1500], 4, 128, extra=1200)
        Q = [c.queries(8, 2.0).cuda() for _ in range(60)]
        new = [torch.randn(4, 1 + i % 40, 4, 128, generator=c.g).bfloat16().cuda() for i in range(60)]
        ws = [tr.workspace(x) for x in (tr.tr_kv_append_workspace_bytes(c.cache),
                                        tr.tr_decode_attn_workspace_bytes(c.cache, 8, True),
                                        tr.tr_kv_evict_workspace_bytes(c.cache, 600))]
        O = [torch.empty(4, 8, 128, device="cuda") for _ in range(60)]
        pause = torch.cuda.synchronize if wait else lambda: None
        pause()
        for i in range(60):
            tr.tr_kv_append(new[i], new[i], c.cache, ws[0])
            pause()
            tr.tr_decode_attn(Q[i], c.cache, O[i], 0.09, ws[1], accumulate=True)
            pause()
            if i % 3 == 2:
                tr.tr_kv_evict(c.cache, 600, 100, ws[2])
                pause()
        torch.cuda.synchronize()
        outs.append(O + [c.scores, c.L, raw(c.K), raw(c.V)])
    assert all(torch.equal(x, y) for x, y in zip(*outs))


@pytest.mark.parametrize("type,layout", [("bf16", "dense"), ("bf16", 16), ("e4m3", 16), ("f16", "nhd4")])
def test_decoding_steps_with_eviction(tr, type, layout):
    """Prompt, then steps of append + attention with weights gathered, cut back whenever a sequence passes 48 rows;
    a host model that keeps the same rows follows every step."""
    rng = np.random.default_rng(40)
    c = Made(tr, rng, type, layout, [0, 0, 0], 2, 64, extra=96)
    check_append(c, 40, [40, 13, 0])
    for step in range(30):
        check_append(c, 1 + step % 3, None)
        Q = c.queries(6, 2.0)
        # NaN that an 8-bit append was tested with must not take part
        if type == "e4m3":
            for b in range(3):
                for x, rows in ((c.K, c.rows_k), (c.V, c.rows_v)):
                    rows[b] = torch.nan_to_num(rows[b].float(), 0.0).to(TYPES["e4m3"])
                    c.put(x, b, rows[b])
        before = c.scores.clone()
        O, lse = c.attend(Q, 0.125, accumulate=True)
        c.check(Q, 0.125, O, lse, before)
        if max(c.lengths) > 48:
            check_evict(c, 32, 8)


def test_scores_behind_an_eviction_and_commits_of_tree_steps(tr):
    """An eviction leaves scores behind the budget as they are and a tree step's commit does not touch them: set to 0
    in between, as the header asks, the committed rows start from nothing."""
    B, Hkv, cap, d, budget = 2, 2, 96, 128, 24
    c = Made(tr, np.random.default_rng(55), "bf16", "dense", [60, 41], Hkv, d, extra=36)
    assert c.cap == cap
    tr.tr_kv_evict(c.cache, budget, 4, tr.workspace(tr.tr_kv_evict_workspace_bytes(c.cache, budget)))
    left = c.scores.clone()
    assert bool((left[0, :, budget:60] > 0).all())
    c.scores[:, :, budget:].zero_()
    tree = tr.Tree((2, 1, 0, 0), 4)
    kt = torch.randn(B, tree.N, Hkv, d, generator=c.g).bfloat16().cuda()
    path = torch.tensor([[0, 1, 3], [0, 2, 0]], dtype=torch.int32, device="cuda")
    acc = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    tr.tr_kv_commit(kt, kt, c.K, c.V, c.L, tree, path, acc, tr.workspace(tr.tr_kv_commit_workspace_bytes(B)))
    assert c.L.tolist() == [27, 26]
    before = c.scores.clone()
    assert torch.equal(before[:, :, :budget], left[:, :, :budget]) and not before[:, :, budget:].any()
    c.lengths = [27, 26]
    c.rows_k, c.rows_v = [[c.get(x, b, n) for b, n in enumerate(c.lengths)] for x in (c.K, c.V)]
    Q = c.queries(4, 2.0)
    O, lse = c.attend(Q, 0.09, accumulate=True)
    c.check(Q, 0.09, O, lse, before)


@pytest.mark.parametrize("budget", [0, 100])
def test_engine_alternates_tree_and_single_token_steps(tr, budget):
    """TRState: tree steps and steps without a draft on one state, evictions between them, against the oracle's loop
    (a step without a draft is the loop's step on a one-node tree); the committed tokens are plain greedy decoding."""
    import synth
    from free_speculative_decoding_gb300.engine import TRState
    from gpu_util import ATTN_TOL, gpu_start, oracle_qkv, oracle_states, rows_rel_err, target_fn
    from synth import device as sd

    w = synth.WORKLOADS["tiny"].scaled(prefix=(100, 140), B=2, Hq=8, Hkv=4, V=5000, steps=24)
    tree, plan, plan1 = tr.Tree(w.child_counts, w.K), oracle.TreePlan(w.child_counts, w.K), oracle.TreePlan((0,), w.K)
    st = TRState(tree, w.B, w.V, Hq=w.Hq, Hkv=w.Hkv, d=w.d, cap=w.capacity(), single_token=True, budget=budget,
                 recent=20 if budget else 0)
    sd.fill_cache(w, st)
    gpu_start(w, st)
    states, target, qkv = oracle_states(w), target_fn(w), oracle_qkv(w)
    tgt, logits1 = sd.DeviceTarget(w, tree), torch.empty(w.B, w.V, device="cuda")
    gathered = [np.zeros((w.Hkv, w.capacity())) for _ in range(w.B)]
    evicted = 0
    for s in range(w.steps):
        q, kt, vt = sd.step_qkv(w, s, tree.N)
        plain, recs = s % 3 != 0, {}
        before = [(x.kc.copy(), x.vc.copy(), x.L) for x in states]
        qo, ko, vo = qkv(s)
        one = (qo[:, :1], ko[:, :1], vo[:, :1]) if plain else (qo, ko, vo)
        oracle.tr_loop(plan1 if plain else plan, states, target, 1, w.K, qkv=lambda _: one, scale=w.d ** -0.5,
                       on_step=lambda _, b, rec: recs.__setitem__(b, rec))
        if plain:
            tr.trsyn_logits(w.seed, st.tree1, st.root.unsqueeze(1), st.L, logits1)
            O = st.decode(q[:, 0].contiguous(), kt[:, 0].contiguous(), vt[:, 0].contiguous())
            got_O = O.cpu().numpy()[:, None]
            st.finish_decode(logits1)
            for b in range(w.B):
                kc, vc, L = before[b]
                kc[:, L], vc[:, L] = ko[b, 0], vo[b, 0]
                _, _, W = oracle.decode_attention(qo[b, 0], kc[:, :L + 1], vc[:, :L + 1], w.d ** -0.5)
                gathered[b][:, :L + 1] += W.reshape(w.Hkv, -1, L + 1).sum(1)
                assert st.committed1[b].tolist() == recs[b]["committed"]
        else:
            got_O = st.verify(q, kt, vt).cpu().numpy()
            st.finish(logits=tgt.logits_for(st), Kt=kt, Vt=vt)
        for b in range(w.B):
            assert rows_rel_err(got_O[b], recs[b]["O"]) <= ATTN_TOL
            assert st.acc_len[b].item() == recs[b]["acc_len"]
            assert np.array_equal(st.M[b].cpu().numpy(), states[b].M)
            assert st.root[b].item() == states[b].root and st.L[b].item() == states[b].L
            assert np.array_equal(st.tree_tok[b].cpu().numpy(), oracle.retrieve(states[b].M, states[b].root, plan))
        if budget:
            sc = st.scores.cpu().numpy()
            for b in range(w.B):
                assert np.allclose(sc[b], gathered[b], rtol=1e-5, atol=1e-7)
            if s % 5 == 4:
                lens = [x.L for x in states]
                st.evict()
                for b, x in enumerate(states):
                    if x.L > budget:
                        evicted += 1
                        for h in range(w.Hkv):
                            keep = oracle.evict_keep(sc[b, h, :x.L], budget, 20)
                            for t in (x.kc, x.vc):
                                t[h, :budget] = t[h, keep]
                            gathered[b][h, :budget] = sc[b, h, keep]
                        x.L = budget
                    gathered[b][:, x.L:] = 0
                    assert st.L[b].item() == min(lens[b], budget)
    assert not budget or evicted >= 4
    if not budget:
        L0, roots = w.prefix_lengths(), synth.initial_roots(w)
        for b in range(w.B):
            out = states[b].emitted
            top1 = lambda pos, tok: np.argmax(target(b, np.array([pos]), np.array([tok]))[0])
            assert out == oracle.greedy_decode(top1, int(roots[b]), int(L0[b]), len(out))
    with pytest.raises(ValueError):
        TRState(tree, 1, 100, budget=5)
    if not budget:
        with pytest.raises(ValueError, match="budget"):
            st.evict()
