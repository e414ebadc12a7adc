"""Sampling with temperature, top-k, top-p and min-p on the GPU against the 64-bit oracle
(GB300 only).

A draw has to be the oracle's token wherever the uniform, and the sum at top-p's edge, are
further from a border than the arithmetic can move it: the weights are off by 2^-29, relative,
at most (the fraction's power of two: a table rounded to 2^-31, a polynomial whose value is below 2^-7
in fp32 steps of 2^-31, one rounding to 2^-31; the exponent is good to 2^-33), so a sum's share of
another by 2^-28.  Weights are whole numbers of a unit of 2^-S, S = 62 - floor(log2 V) > 61 - log2 V, and the largest
is 2^(S - t), 0 <= t <= 1.02.  A cut to a whole number takes less than one unit from a token, and one whose weight is
below 2^-(S - 2) of the largest, so of 2^(2 - t) units at most, counts as none.  The V tokens lose at most
max(V, V 2^(2 - t)) units of a sum that is at least 2^(S - t): below V 2^(2 - S) < V^2 2^-59 of it (the one-unit
cuts: V 2^(1.02 - S), less than that).  Rows nearer than that are counted and must be rare.  ln(w / W) is off by 2^-28 + that and
fp32's half step of it (and of a double's log)."""
import math

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
    assert torch.cuda.get_device_capability() == (10, 3)
    return m


@pytest.fixture(autouse=True)
def status_stays_clean(tr):
    yield
    assert tr.tr_get_status() == 0


def near(V):
    return 2.0 ** -28 + V * V * 2.0 ** -59


def draw(tr, x, U, V=None, **rules):
    rows = x.shape[0]
    cu = lambda v, t: None if v is None else torch.as_tensor(v, dtype=t).cuda()
    token = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((rows,), 7.0, device="cuda")
    tr.tr_sample(x, cu(U, torch.float32), token, temperature=cu(rules.get("temperature"), torch.float32),
                 top_k=cu(rules.get("top_k"), torch.int32), top_p=cu(rules.get("top_p"), torch.float32),
                 min_p=cu(rules.get("min_p"), torch.float32), logprob=lp, V=V)
    return token.cpu().numpy(), lp.cpu().numpy()


def check(tr, x, U, V=None, most_near=0.01, **rules):
    """x [rows, ld] on the GPU; rules: a list for each rule."""
    n = x.shape[1] if V is None else V
    token, lp = draw(tr, x, U, V, **rules)
    host = x[:, :n].float().cpu().numpy().astype(np.float64)
    at_border = 0
    for r in range(x.shape[0]):
        f = lambda k, off: off if rules.get(k) is None else float(np.float32(rules[k][r]))
        kw = dict(temperature=f("temperature", 1.0), top_k=int(f("top_k", 0)), top_p=f("top_p", 1.0), min_p=f("min_p", 0.0))
        t, l, margin = oracle.sample(host[r], float(np.float32(U[r])), **kw)
        if token[r] != t:
            # only next to a border, and a token that the oracle could draw there
            assert margin <= near(n), (r, kw, token[r], t, margin)
            at_border += 1
            continue
        if margin > near(n):
            tol = 2 * near(n) + 2.0 ** -23 * abs(l) + 2.0 ** -149
            assert (lp[r] == l) if math.isinf(l) else abs(lp[r] - l) <= tol, (r, kw, lp[r], l)
    assert at_border <= most_near * x.shape[0] + (1 if x.shape[0] > 20 else 0)
    return token


def logits(rows, ld, spread, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(rows, ld, device="cuda").normal_(generator=g) * spread
    at = torch.randint(ld, (rows, 8), device="cuda", generator=g)
    x.scatter_add_(1, at, torch.full((rows, 8), 3.0 * spread, device="cuda"))
    return x.to(dtype)


def uniforms(rng, rows):
    return np.float32(rng.random(rows)).tolist()


RULES = {
    "none": lambda rng, n: {},
    "temperature": lambda rng, n: dict(temperature=(0.2 + 2 * rng.random(n)).tolist()),
    "top_k": lambda rng, n: dict(top_k=rng.integers(0, 60, n).tolist(), temperature=[0.8] * n),
    "top_p": lambda rng, n: dict(top_p=rng.random(n).tolist(), temperature=(0.2 + rng.random(n)).tolist()),
    "min_p": lambda rng, n: dict(min_p=(0.3 * rng.random(n)).tolist()),
    "all": lambda rng, n: dict(temperature=np.where(rng.random(n) < 0.1, 0, 0.2 + rng.random(n)).tolist(),
                               top_k=np.where(rng.random(n) < 0.4, 0, np.exp(rng.random(n) * 9).astype(int)).tolist(),
                               top_p=np.where(rng.random(n) < 0.3, 1.0, rng.random(n)).tolist(),
                               min_p=np.where(rng.random(n) < 0.5, 0.0, 0.2 * rng.random(n)).tolist()),
}


@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("V", [1, 2, 3, 31, 32, 33, 511, 512, 513, 1000, 4099])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_rows(tr, rule, V, dtype):
    rng = np.random.default_rng(V)
    n = 40
    for pad, spread in ((0, 1.0), (3, 3.0)):
        check(tr, logits(n, V + pad, spread, dtype, V + pad), uniforms(rng, n), V, **RULES[rule](rng, n))


@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("V,ld,dtype,spread", [(32000, 32000, torch.float32, 1.0), (50257, 50257, torch.float32, 2.0),
                                               (50257, 50261, torch.bfloat16, 1.0), (128256, 128256, torch.bfloat16, 2.0),
                                               (128256, 128256, torch.float32, 3.0), (131071, 131072, torch.float32, 0.1)])
def test_vocabularies(tr, rule, V, ld, dtype, spread):
    rng = np.random.default_rng(V)
    check(tr, logits(24, ld, spread, dtype, 5), uniforms(rng, 24), V, **RULES[rule](rng, 24))


@pytest.mark.parametrize("rule", ["none", "top_p", "all"])
@pytest.mark.parametrize("V", [400_003, 1_000_000, 3_000_001])
def test_rows_larger_than_the_chip_holds(tr, rule, V):
    rng = np.random.default_rng(V)
    check(tr, logits(3, V, 2.0, torch.float32, 6), uniforms(rng, 3), **RULES[rule](rng, 3))


@pytest.mark.parametrize("rows", [1, 2, 37, 152, 153, 305, 1280, 5000])
def test_row_counts(tr, rows):
    rng = np.random.default_rng(rows)
    check(tr, logits(rows, 600, 2.0, torch.float32, rows), uniforms(rng, rows), **RULES["all"](rng, rows))


@pytest.mark.parametrize("V", [4, 64, 1024, 32768, 262144])
@pytest.mark.parametrize("value", [0.0, -7.25, 1e30])
def test_equal_logits_draw_exactly(tr, V, value):
    """V equal weights: the token is floor(U V') of the V' that the rules leave, exactly, on the borders too."""
    n = 64
    x = torch.full((n, V), value, device="cuda")
    u = [i / n for i in range(n)]
    token, lp = draw(tr, x, u)
    assert token.tolist() == [int(i * V // n) for i in range(n)] and np.allclose(lp, -math.log(V), rtol=1e-6)
    below = [np.nextafter(np.float32(i + 1) / np.float32(n), np.float32(0)).item() for i in range(n)]
    token, _ = draw(tr, x, below)
    assert token.tolist() == [min(int(b * V), V - 1) for b in below]
    # ties leave the lowest IDs: half of them by top-p (reached exactly), k of them by top-k
    half = draw(tr, x, u, top_p=[0.5] * n)[0]
    assert half.tolist() == [int(i * (V // 2) // n) for i in range(n)]
    k = [max(V // 4, 1)] * n
    assert draw(tr, x, u, top_k=k)[0].tolist() == [int(i * k[0] // n) for i in range(n)]
    assert draw(tr, x, u, top_k=k, top_p=[0.25] * n)[0].tolist() == [int(i * max(math.ceil(k[0] / 4), 1) // n) for i in range(n)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [700, 40001])
def test_heavy_ties(tr, dtype, V):
    """A handful of values: edges fall inside long runs of equal logits."""
    rng = np.random.default_rng(V)
    g = torch.Generator().manual_seed(V)
    x = (torch.randint(-2, 3, (60, V), generator=g) / 2).to(dtype).cuda()
    x[::7, V // 3] = 9.0
    for rule in ("top_k", "top_p", "all"):
        r = RULES[rule](rng, 60)
        if "top_k" in r:
            r["top_k"] = rng.integers(1, V + 5, 60).tolist()
        check(tr, x, uniforms(rng, 60), most_near=0.05, **r)


def test_masked_and_special_logits(tr):
    inf, nan = math.inf, math.nan
    rng = np.random.default_rng(3)
    V, n = 3001, 48
    x = logits(n, V, 2.0, torch.float32, 9)
    g = torch.Generator(device="cuda").manual_seed(1)
    x[torch.rand(n, V, device="cuda", generator=g) < 0.6] = -inf
    x[:, 5::17] = nan
    x[3, :] = -inf                       # nothing is left
    x[4, :] = nan
    x[5, :], x[5, 2900] = -inf, -3e38    # one token
    x[6, 7], x[6, 2000] = inf, inf       # these two share the draw
    x[7, :] = -3.4e38                    # differences that pass fp32's range
    x[7, 10] = 3.4e38
    x[8, :], x[8, 0], x[8, 1] = -inf, 0.0, -0.0
    x[9, :] = torch.linspace(-1e-40, 1e-40, V)   # denormal numbers
    for rule in RULES:
        r = RULES[rule](rng, n)
        token = check(tr, x, uniforms(rng, n), **r)
        assert token[3] == -1 and token[4] == -1 and token[5] == 2900 and token[6] in (7, 2000) and token[8] in (0, 1)
    bf = x.bfloat16()
    check(tr, bf, uniforms(rng, n), **RULES["all"](rng, n))


def test_parameters_at_their_ends(tr):
    inf, nan = math.inf, math.nan
    rng = np.random.default_rng(4)
    temps = [0.0, -1.0, nan, 1e-45, 2.0 ** -126, 1e-20, 1e-3, 1.0, 50.0, 3e38, inf]
    ks = [0, -5, 1, 2, 499, 500, 501, 2 ** 31 - 1, -2 ** 31]
    ps = [nan, -1.0, 0.0, 1e-45, 1e-30, 1e-7, 0.5, 1 - 2.0 ** -24, 1.0, 2.0, inf]
    ms = [nan, -1.0, 0.0, 1e-45, 1e-30, 0.5, 1.0, 1.5, inf]
    us = [0.0, 1 - 2.0 ** -24, 1.0, -0.5, nan, 2.0 ** -149, 1e-30, 0.5, inf, -inf]
    n = 600
    pick = lambda v: [v[i] for i in rng.integers(0, len(v), n)]
    x = logits(n, 500, 1.5, torch.float32, 8)
    check(tr, x, pick(us), temperature=pick(temps), top_k=pick(ks), top_p=pick(ps), min_p=pick(ms))
    for name, values in (("temperature", temps), ("top_k", ks), ("top_p", ps), ("min_p", ms)):
        v = pick(values)
        check(tr, x, pick(us), **{name: v})


def test_draws_follow_the_distribution(tr):
    """Evenly spaced uniforms: every token is drawn as often as its probability says, to within one draw."""
    V, n = 300, 4096
    x = logits(1, V, 1.0, torch.float32, 2)
    U = [(i + 0.5) / n for i in range(n)]
    token, lp = draw(tr, x.expand(n, V).contiguous(), U, temperature=[0.7] * n, top_p=[0.9] * n)
    ids, w, _ = oracle.sample_left(x[0].cpu().numpy(), float(np.float32(0.7)), 0, float(np.float32(0.9)))
    p = np.zeros(V)
    p[ids] = w / w.sum()
    assert np.abs(np.bincount(token, minlength=V) - n * p).max() <= 1.0 + 1e-5
    assert np.allclose(lp, np.log(p[token]), rtol=1e-6)


def test_equal_calls_give_equal_bits(tr):
    rng = np.random.default_rng(6)
    x = logits(64, 128256, 1.0, torch.float32, 3)
    u, r = uniforms(rng, 64), RULES["all"](rng, 64)
    a, b = draw(tr, x, u, **r), draw(tr, x, u, **r)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1].view(np.int32), b[1].view(np.int32))


def test_one_row_alone_and_among_others(tr):
    """The launch goes by the number of rows; a row's result does not."""
    rng = np.random.default_rng(7)
    for V, dtype in ((32000, torch.float32), (128256, torch.bfloat16), (50257, torch.float32)):
        x = logits(600, V, 1.0, dtype, 4)
        u, r = uniforms(rng, 600), RULES["all"](rng, 600)
        token, lp = draw(tr, x, u, **r)
        for i in (0, 1, 77, 599):
            for m in (1, 5, 40):
                lo = min(i, 600 - m)
                t, l = draw(tr, x[lo:lo + m], u[lo:lo + m], **{k: v[lo:lo + m] for k, v in r.items()})
                assert np.array_equal(t, token[lo:lo + m]) and np.array_equal(l.view(np.int32), lp[lo:lo + m].view(np.int32))


def test_rows_past_2_31_elements(tr):
    V, n = 262144, 8200
    x = torch.empty(n, V, dtype=torch.bfloat16, device="cuda")
    x[:] = logits(1, V, 1.0, torch.bfloat16, 3)
    x[-1] = logits(1, V, 1.0, torch.bfloat16, 4)[0]
    token, _ = draw(tr, x, [0.37] * n, top_p=[0.8] * n)
    assert (token[:-1] == token[0]).all()
    check(tr, x[-3:].contiguous(), [0.37] * 3, top_p=[0.8] * 3)
    assert oracle.sample(x[-1].float().cpu().numpy(), float(np.float32(0.37)), top_p=float(np.float32(0.8)))[0] == token[-1]


def test_in_a_graph_on_another_stream(tr):
    rng = np.random.default_rng(8)
    n, V = 20, 9000
    x = logits(n, V, 1.0, torch.float32, 1)
    U, T, p = (torch.rand(n, device="cuda") for _ in range(3))
    k = torch.randint(0, 50, (n,), dtype=torch.int32, device="cuda")
    token = torch.zeros(n, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            tr.tr_sample(x, U, token, temperature=T, top_k=k, top_p=p)
        for rep in range(3):
            x.mul_(1.5)
            U.uniform_()
            T.uniform_(0.3, 2.0)
            g.replay()
            s.synchronize()
            want, _ = draw(tr, x, U, temperature=T, top_k=k, top_p=p)
            assert np.array_equal(token.cpu().numpy(), want)
            check(tr, x, U.tolist(), temperature=T.tolist(), top_k=k.tolist(), top_p=p.tolist())
    torch.cuda.current_stream().wait_stream(s)


def test_binding_refuses(tr):
    x = torch.zeros(4, 10, device="cuda")
    U, token = torch.zeros(4, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    tr.tr_sample(x, U, token)
    for kw in (dict(x=x[0]), dict(x=x.half()), dict(x=x.cpu()), dict(x=x.t()), dict(U=U[:3]), dict(U=U.double()), dict(U=U.cpu()),
               dict(token=token.long()), dict(token=token[:2]), dict(temperature=U[:1]), dict(top_k=U), dict(top_p=token),
               dict(min_p=U.half()), dict(logprob=token), dict(logprob=U[:3]), dict(V=-1), dict(V=1 << 32),
               dict(U=torch.zeros(8, device="cuda")[::2])):
        a = dict(x=x, U=U, token=token)
        a.update(kw)
        with pytest.raises(ValueError):
            tr.tr_sample(a.pop("x"), a.pop("U"), a.pop("token"), **a)
    for V in (11, 0):
        with pytest.raises(tr.TRError):
            tr.tr_sample(x, U, token, V=V)
    empty = torch.zeros(0, 10, device="cuda")
    tr.tr_sample(empty, U[:0], token[:0])


# Where a launch changes its shape: a CTA's slice that fills shared memory (192 KB alone, 88 KB shared) in a
# cluster of eight, and one granule more; rows from which CTAs share an SM, and from which there are more of them.
@pytest.mark.parametrize("rows,V,dtype", [
    (1, 8 * 48 * 1024, torch.float32), (1, 8 * 48 * 1024 + 5, torch.float32), (2, 8 * 96 * 1024 + 1, torch.bfloat16),
    (19, 32003, torch.float32), (20, 32003, torch.float32), (38, 180223, torch.float32), (39, 180223, torch.float32),
    (30, 180225, torch.float32), (30, 360447, torch.bfloat16), (30, 360451, torch.bfloat16), (76, 45000, torch.float32),
    (152, 22529, torch.float32), (304, 22528, torch.float32), (305, 22528, torch.float32), (77, 90001, torch.float32)])
def test_shapes_of_a_launch(tr, rows, V, dtype):
    rng = np.random.default_rng(rows + V)
    x = logits(rows, V + 3, 1.5, dtype, rows)
    r = RULES["all"](rng, rows)
    check(tr, x, uniforms(rng, rows), V, **r)
    flat = x.view(-1)[1:1 + (rows - 1) * V].view(rows - 1, V) if rows > 1 else None  # rows that start anywhere
    if flat is not None:
        check(tr, flat, uniforms(rng, rows - 1), V, **{k: v[1:] for k, v in r.items()})


@pytest.mark.parametrize("rows,V", [(1, 40000), (6, 32000), (200, 32000)])
def test_more_tokens_at_the_edge_than_a_list_holds(tr, rows, V):
    """k and p whose edges lie among thousands of equal logits, or of ones that share a histogram's bin."""
    rng = np.random.default_rng(V + rows)
    g = torch.Generator(device="cuda").manual_seed(rows)
    steps = torch.randint(0, 4, (rows, V), device="cuda", generator=g).float()            # four values
    close = 1e-4 * torch.empty(rows, V, device="cuda").normal_(generator=g)                # a narrow range ...
    close[:, 17] = 60.0                                                                    # ... far below one token
    for x in (steps, close):
        for k in (2, 700, 1023, 1024, 1025, 5000, V - 1):
            check(tr, x, uniforms(rng, rows), top_k=[k] * rows, temperature=[30.0] * rows)
            check(tr, x, uniforms(rng, rows), top_k=[k] * rows, top_p=[0.6] * rows, temperature=[30.0] * rows)
        for p in (0.01, 0.5, 0.999):
            check(tr, x, uniforms(rng, rows), top_p=[p] * rows, temperature=[30.0] * rows)


def test_calls_on_two_streams_at_once(tr):
    """Nothing is shared between calls: eight of each kind under way at a time draw what they draw alone."""
    rng = np.random.default_rng(12)
    calls = []
    for i, (rows, V, dtype) in enumerate([(1, 32000, torch.float32), (40, 50257, torch.float32), (700, 20000, torch.bfloat16),
                                          (6, 128256, torch.bfloat16)] * 2):
        x = logits(rows, V, 1.0, dtype, i)
        r = RULES["all"](rng, rows)
        cu = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda") for k, v in r.items()}
        U = torch.tensor(uniforms(rng, rows), device="cuda")
        calls.append((x, U, cu, [torch.full((rows,), -7, dtype=torch.int32, device="cuda") for _ in range(2)]))
    for x, U, r, token in calls:
        tr.tr_sample(x, U, token[0], **r)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for rep in range(5):
        for i, (x, U, r, token) in enumerate(calls):
            with torch.cuda.stream(streams[(i + rep) % 4]):
                tr.tr_sample(x, U, token[1], **r)
        torch.cuda.synchronize()
        for _, _, _, token in calls:
            assert torch.equal(token[0], token[1])
            token[1].fill_(-7)


def test_draws_one_behind_the_other(tr):
    """A call's tokens feed the next call's logits without a wait in between, in a graph and without."""
    n, V = 24, 32000
    table = logits(512, V, 1.0, torch.float32, 21)
    U = torch.rand(6, n, device="cuda")
    p = torch.full((n,), 0.8, device="cuda")

    def run(token, x):
        for step in range(6):
            torch.index_select(table, 0, (token % 512).long(), out=x)
            tr.tr_sample(x, U[step], token, top_p=p)
    token, x = torch.arange(n, dtype=torch.int32, device="cuda"), torch.empty(n, V, device="cuda")
    want = token.clone()
    for step in range(6):
        y = table[(want % 512).long()]
        torch.cuda.synchronize()
        tr.tr_sample(y, U[step], want, top_p=p)
        torch.cuda.synchronize()
    run(token, x)
    assert torch.equal(token, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(token, x)
    for _ in range(3):
        token.copy_(torch.arange(n))
        g.replay()
        assert torch.equal(token, want)


def test_longest_row(tr):
    """2^30 equal logits, the most that a row may have: every draw is known exactly."""
    V = 1 << 30
    x = torch.zeros(1, V, dtype=torch.bfloat16, device="cuda")
    for u in (0.0, 0.37, 1 - 2.0 ** -24):
        for left, rules in ((V, {}), (V >> 1, dict(top_p=[0.5])), (12345, dict(top_k=[12345])), (50, dict(top_k=[50])),
                            (V, dict(min_p=[0.5]))):
            token, lp = draw(tr, x, [u], **rules)
            want = int(float(np.float32(u)) * left)  # exact in 64 bits: 24 + 30 bits
            assert token[0] == want, (u, rules, token[0], want)
            assert abs(lp[0] + math.log(left)) <= 2.0 ** -23 * math.log(left)   # equal whole weights: fp32's half step of the log
