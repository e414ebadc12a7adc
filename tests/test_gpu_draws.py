"""Draws next to borders on the GPU (GB300 only): whatever the uniform, the token is one that the rules
leave, and its stretch of the running sum is where the uniform points, within what the sums may be off.

That is tol = 2^-28 + V^2 2^-59 of a sum, as tests/test_gpu_sample.py derives it for whole weights: every weight is off
by 2^-29, relative, and V of them, each cut to a whole number of units or, below four units, left out, by V 2^(2 - S) of the
largest.  Rows with a temperature alone that are read from global memory are summed in the first pass, in
units of the warp's largest logit so far.  A token then loses one unit to its cut, two at most go with every lane's
rescaled sum (each rescale that shifts by a bit or more loses less than one unit, and every later one
halves that) and one with the warp's; a lane has four tokens and more, a warp 128, so that a token loses less than 1.6 units
of a sum of at least 2^(S - 1.02): below V 2^(2 - S) again, and one that ends below four units is in a sum with as many or with none."""
import math

import numpy as np
import pytest
import torch

import oracle
from test_gpu_sample import RULES, logits

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


def near(V):
    return 2.0 ** -28 + V * V * 2.0 ** -59


def draw(tr, x, U, V=None, **rules):
    cu = lambda v, t: None if v is None else torch.as_tensor(v, dtype=t).cuda()
    token = torch.full((x.shape[0],), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((x.shape[0],), 7.0, device="cuda")
    types = dict(top_k=torch.int32)
    tr.tr_sample(x, cu(U, torch.float32), token, logprob=lp, V=V,
                 **{k: cu(v, types.get(k, torch.float32)) for k, v in rules.items()})
    return token.cpu().numpy(), lp.cpu().numpy()


def check(tr, x, U, V=None, logprobs=False, rows=None, **rules):
    """Every drawn token (of `rows`) is one that may be drawn."""
    n = x.shape[1] if V is None else V
    token, lp = draw(tr, x, U, V, **rules)
    host = x[:, :n].float().cpu().numpy().astype(np.float64)
    off = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    for r in range(x.shape[0]) if rows is None else rows:
        kw = {k: float(np.float32(rules[k][r])) if k in rules else o for k, o in off.items()}
        kw["top_k"] = int(kw["top_k"]) if "top_k" not in rules else int(rules["top_k"][r])
        got = oracle.sample_may_draw(host[r], token[r], float(np.float32(U[r])), near(n), **kw)
        assert got is not None, (r, kw, U[r], token[r], oracle.sample(host[r], float(np.float32(U[r])), **kw))
        assert token[r] == -1 or host[r, token[r]] > -np.inf
        if logprobs and token[r] >= 0:  # off by a weight's and the sum's error, and fp32's half step of it
            e = 2 * near(n) + 2.0 ** -23 * max(abs(got[0]), abs(got[1])) + 2.0 ** -149
            assert got[0] - e <= lp[r] <= got[1] + e, (r, kw, U[r], token[r], lp[r], got)
    return token, lp


# Rows that are read from global memory (more of them than the chip holds at once, or longer ones), and held ones.
@pytest.mark.parametrize("rows,V,dtype", [(200, 32000, torch.float32), (1, 32000, torch.float32), (400, 3001, torch.float32),
                                          (160, 100003, torch.bfloat16), (2, 1000000, torch.float32)])
def test_a_masked_token_is_not_drawn_where_the_first_weights_are_tiny(tr, rows, V, dtype):
    """The first token is masked, and its range holds weights around the least that count: relative to that range's own
    largest logit they are all large."""
    S = 62 - int(math.log2(V))
    x = torch.full((rows, V), -math.inf, device="cuda")
    far = -(S - 2) * math.log(2.0)
    levels = torch.linspace(-1.5, 1.5, rows, device="cuda") if rows > 1 else torch.full((1,), -0.3, device="cuda")
    n = min(4096, V // 2)
    x[:, 1:n] = (far + levels).unsqueeze(1)
    x[:, 20000 % V] = 0.0
    x = x.to(dtype)
    for u in (0.0, 2.0 ** -149, -1.0, math.nan):
        token, _ = check(tr, x, [u] * rows, rows=range(0, rows, 7))
        assert (token > 0).all()
        assert (x[torch.arange(rows), torch.from_numpy(token).long().cuda()] > -math.inf).all()


def steps(kind, rows, V, rng):
    """Logits in units of T."""
    i = np.arange(V) / V
    if kind == "rising":
        x = np.stack([s * (i - 1) for s in rng.choice([0.5, 5.0, 50.0, 2000.0], rows)]) + 0.1 * rng.random((rows, V))
    elif kind == "falling":
        x = np.stack([-s * i for s in rng.choice([0.5, 5.0, 50.0, 2000.0], rows)]) + 0.1 * rng.random((rows, V))
    elif kind == "jumps":   # of more than 63 powers of two, and of less
        at = np.sort(rng.integers(0, V, (rows, 6)), axis=1)
        x = sum((np.arange(V)[None] >= at[:, k:k + 1]) * rng.choice([0.0, 3.0, 30.0, 60.0, 200.0], (rows, 1)) for k in range(6))
        x = x + rng.random((rows, V))
    elif kind == "tails":   # all around the least weight that counts but a few tokens
        x = -(60 - int(math.log2(V))) * math.log(2.0) + rng.normal(size=(rows, V))
        x[np.arange(rows)[:, None], rng.integers(0, V, (rows, 3))] = 0.0
    else:                   # masked
        x = 4.0 * rng.normal(size=(rows, V))
        x[rng.random((rows, V)) < 0.7] = -np.inf
        x[:, 3::11] = np.nan
    return x


@pytest.mark.parametrize("kind", ["rising", "falling", "jumps", "tails", "masked"])
@pytest.mark.parametrize("rows,V,dtype", [(170, 32000, torch.float32), (400, 3001, torch.float32), (310, 5003, torch.bfloat16),
                                          (4, 500003, torch.float32)])
def test_temperature_alone(tr, kind, rows, V, dtype):
    """Sums that are rescaled as the largest logit rises: T from 0.2 to 2 over many rows, and the same rows a few at a time."""
    rng = np.random.default_rng(V + rows)
    T = np.float32(0.2 + 1.8 * rng.random(rows))
    x = torch.from_numpy(steps(kind, rows, V, rng) * T[:, None]).to(dtype).cuda()
    U = np.float32(rng.random(rows))
    U[::5], U[1::5], U[2::10] = 0.0, np.float32(1 - 2.0 ** -24), np.float32(2.0 ** -149)
    some = range(rows) if V < 10000 else range(0, rows, 4)
    check(tr, x, U.tolist(), rows=some, temperature=T.tolist())
    check(tr, x[:3].contiguous(), U[:3].tolist(), temperature=T[:3].tolist())


@pytest.mark.parametrize("rows,V,dtype", [(9, 3000, torch.float32), (400, 3001, torch.float32), (170, 32000, torch.bfloat16)])
@pytest.mark.parametrize("rules", [dict(), dict(top_k=2000), dict(top_p=1 - 2.0 ** -24), dict(min_p=1e-30)])
def test_log_probabilities_of_tiny_weights(tr, rows, V, dtype, rules):
    """U = 0 draws the first token that has weight, down to four units of 2^-S: its logarithm keeps fp32's precision although
    the whole number of units does not."""
    rng = np.random.default_rng(rows)
    S = 62 - int(math.log2(V))
    T = np.float32(0.3 + rng.random(rows))
    level = np.linspace(0.0, (S - 3.2) * math.log(2.0), rows)
    x = np.full((rows, V), -np.inf)
    x[:, 3] = -level
    x[:, 50:1000] = -0.5 * rng.random((rows, 950))
    x[:, 1700] = 0.0
    x = (x * T[:, None] + rng.choice([0.0, -300.0, 2.0 ** 21], (rows, 1)) * (dtype is torch.float32))
    x = torch.from_numpy(np.float32(x)).to(dtype).cuda()
    x[rows // 2, 3:] = x[rows // 2, 3].clone()     # equal ones
    token, _ = check(tr, x, [0.0] * rows, logprobs=True, temperature=T.tolist(), **{k: [v] * rows for k, v in rules.items()})
    if not rules:
        assert (token == 3).mean() > 0.9


# What tests/test_gpu_sample.py compares away from borders, next to them: there it asks only that a border is near.
ENDS = [0.0, 1 - 2.0 ** -24, 1.0, -0.5, math.nan, 2.0 ** -149, 2.0 ** -30, 1e-9, 0.5]


@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("rows,V,dtype,spread", [
    (54, 33, torch.float32, 1.0), (54, 512, torch.bfloat16, 6.0), (54, 4099, torch.float32, 6.0), (9, 32000, torch.float32, 4.0),
    (400, 601, torch.float32, 8.0), (180, 32003, torch.float32, 4.0), (45, 128256, torch.bfloat16, 4.0),
    (3, 1000000, torch.float32, 4.0)])
def test_uniforms_at_their_ends(tr, rule, rows, V, dtype, spread):
    rng = np.random.default_rng(V)
    x = logits(rows, V, spread, dtype, V)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x[torch.rand(rows, V, device="cuda", generator=g) < 0.3] = -math.inf
    x[:, 2::9] = math.nan
    x[:, :2] = -math.inf
    U = [ENDS[i % 9] for i in rng.permutation(rows)]
    some = range(rows) if rows * V < 10 ** 6 else range(0, rows, max(1, rows * V // 10 ** 6))
    check(tr, x, U, logprobs=True, rows=some, **RULES[rule](rng, rows))


@pytest.mark.parametrize("rows,V", [(40, 700), (320, 5001), (6, 40001)])
def test_edges_among_equal_logits(tr, rows, V):
    """top-p's mark on a sum of equal weights: the edge may lie on either side of it, no further."""
    rng = np.random.default_rng(V)
    g = torch.Generator().manual_seed(V)
    x = (torch.randint(-2, 3, (rows, V), generator=g) / 2).cuda()
    x[::7, V // 3] = 9.0
    left = [oracle.sample_left(r)[1] for r in x.double().cpu().numpy()]
    p = [float(np.cumsum(np.sort(w)[::-1])[rng.integers(0, V)] / w.sum()) for w in left]
    check(tr, x, rng.random(rows).tolist(), logprobs=True, top_p=p)
    check(tr, x, [1 - 2.0 ** -24] * rows, logprobs=True, top_p=p)
    check(tr, x, rng.random(rows).tolist(), logprobs=True, top_p=p, top_k=rng.integers(1, V, rows).tolist())


def test_a_step_whose_row_leaves_nothing(tr):
    """The root is -1 and the status says so; the other sequence goes on, and so does this one from the next draw."""
    from free_speculative_decoding_gb300.engine import TRState
    V = 500
    tree = tr.Tree((2, 1, 0, 0), 4)
    st = TRState(tree, 2, V, Hq=2, Hkv=1, d=128, cap=64, single_token=True)
    st.start([3, 4], [0, 0], mode=tr.TR_INIT_RANDOM)
    x = torch.randn(2, V, device="cuda")
    x[0] = -math.inf
    U = torch.tensor([0.4, 0.4], device="cuda")
    st.finish_decode(x, U)
    assert tr.tr_get_status() == tr.TR_DEV_BAD_TOKEN
    want = oracle.sample(x[1].double().cpu().numpy(), float(np.float32(0.4)))[0]
    assert st.root.tolist() == [-1, want] and st.committed1.tolist() == [[-1], [want]] and st.tree_tok[1, 0].item() == want
    x[0] = x[1]
    st.finish_decode(x, U)                        # the row of M at the root -1 is not written
    assert tr.tr_get_status() == tr.TR_DEV_BAD_TOKEN and st.root.tolist() == [want, want]
    st.finish_decode(x, U)
    assert tr.tr_get_status() == 0 and st.tree_tok[:, 0].tolist() == [want, want]


@pytest.mark.parametrize("rows", [1, 60, 700])
def test_infinite_logits_at_an_infinite_temperature(tr, rows):
    """The infinite ones share the draw at every temperature."""
    x = torch.randn(rows, 1001, device="cuda")
    x[:, 900] = math.inf
    x[rows // 2:, 17] = math.inf
    U = [i / rows for i in range(rows)]
    for T in (math.inf, 3e38, 1.0):
        for rules in (dict(), dict(top_p=[0.9] * rows), dict(top_k=[5] * rows), dict(min_p=[0.1] * rows)):
            token, lp = check(tr, x, U, logprobs=True, temperature=[T] * rows, **rules)
            assert set(token) <= {17, 900}
