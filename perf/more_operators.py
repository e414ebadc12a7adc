"""The operators on both sides of attention and their cases: norms and position rotation of queries and keys
(tr_qkv_rope), the same on the way into a KV cache (tr_kv_append_rope), and sampling the next token with temperature,
top-k, top-p and min-p from given uniforms (tr_sample).

`run` computes them in plain torch operations in 32 bits (64 for angles and sampling), or, with `own` set, calls the
package's operators."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # one sequence's draft tree, 32 heads: the smallest verification step
        dict(name="rope_1x80_tree", op="rope", type="bf16", B=1, T=80, Hq=32, Hkv=32, d=128, rot=128, pairs=False,
             norm=False, tree=True, far=600),
        # the grouped-query workload: 8 trees of 128 nodes, 32/8 heads, with the norms that such models have
        dict(name="rope_8x128_tree_gqa", op="rope", type="bf16", B=8, T=128, Hq=32, Hkv=8, d=128, rot=128, pairs=False,
             norm=True, tree=True, far=4096),
        # prompts, the largest: four of 8192 tokens
        dict(name="rope_4x8k_prompt", op="rope", type="bf16", B=4, T=8192, Hq=32, Hkv=8, d=128, rot=128, pairs=False,
             norm=True, tree=False, far=1 << 20),
        # a small model: heads of 64, half of them rotated, neighbouring pairs, an odd group, odd lengths
        dict(name="rope_3xodd_f16_d64", op="rope", type="f16", B=3, T=1237, Hq=15, Hkv=5, d=64, rot=32, pairs=True,
             norm=False, tree=False, far=70000),
        # the new token of one sequence: the smallest step a user waits for
        dict(name="append_1x1", op="append", type="bf16", B=1, T=1, Hq=32, Hkv=32, d=128, rot=128, pairs=False,
             norm=False, page=0, lo=512, hi=512, far=0),
        # a serving batch's new tokens, 8-bit cache in small pages, positions that eviction has left behind
        dict(name="append_64x1_e4m3", op="append", type="e4m3", B=64, T=1, Hq=32, Hkv=8, d=128, rot=128, pairs=False,
             norm=True, page=16, lo=1, hi=8191, far=131072),
        # ragged prompts of up to 4096 tokens taken into pages
        dict(name="append_8x4k", op="append", type="bf16", B=8, T=4096, Hq=32, Hkv=8, d=128, rot=128, pairs=False,
             norm=True, page=64, lo=0, hi=300, far=0),
        # a small model's drafts of 33 tokens, odd lengths
        dict(name="append_24x33_f16_d64", op="append", type="f16", B=24, T=33, Hq=15, Hkv=5, d=64, rot=64, pairs=True,
             norm=False, page=32, lo=17, hi=2011, far=0),
        # one sequence's next token under the nucleus rule
        dict(name="sample_1x32000", op="sample", type="f32", rows=1, V=32000, pad=0, spread=1.0, rule="top_p"),
        # a serving batch, every request with rules of its own, the 128k vocabulary
        dict(name="sample_64x128k_mixed", op="sample", type="bf16", rows=64, V=128256, pad=0, spread=2.0, rule="mixed"),
        # every node of the batched workload's trees, rules mixed
        dict(name="sample_1280x32000_mixed", op="sample", type="f32", rows=1280, V=32000, pad=0, spread=1.0,
             rule="mixed"),
        # rows of an odd size, temperature alone
        dict(name="sample_333x50257_plain", op="sample", type="f32", rows=333, V=50257, pad=0, spread=1.5,
             rule="plain"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    while True:
        op = rng.choice(("rope", "append", "sample"))
        if op == "sample":
            c = dict(op=op, type=rng.choice(("f32", "f32", "bf16")), rows=_log(rng, 1, 1280), V=_log(rng, 1000, 262144),
                     pad=rng.choice((0, 0, 1, 8)), spread=rng.choice((1.0, 1.5, 2.0, 3.0)),
                     rule=rng.choice(("plain", "top_k", "top_p", "min_p", "mixed", "mixed")))
            if c["rows"] * c["V"] <= 4.1e7:
                return c
            continue
        c = dict(op=op, type=rng.choice(("bf16", "bf16", "f16") if op == "rope" else ("bf16", "bf16", "f16", "e4m3")),
                 B=_log(rng, 1, 64), T=_log(rng, 1, 8192), Hkv=rng.choice((1, 2, 4, 5, 8, 16, 32)),
                 d=rng.choice((64, 128, 128)), pairs=rng.random() < 0.4, norm=rng.random() < 0.5)
        c["Hq"] = c["Hkv"] * rng.choice((1, 1, 2, 3, 4, 5, 8))
        c["rot"] = rng.choice((c["d"], c["d"], c["d"] // 2, c["d"] // 4))
        c["far"] = rng.choice((0, _log(rng, 1, 1 << 22)))
        if op == "rope":
            c["tree"] = rng.random() < 0.4
            if c["tree"]:
                c["T"] = _log(rng, 1, 128)
        else:
            c["page"] = rng.choice((0, 16, 32, 64, 128, 256))
            if rng.random() < 0.4:
                c["T"] = 1
            c["hi"] = _log(rng, 1, 8192)
            c["lo"] = rng.choice((c["hi"], 0))
        if c["B"] * c["T"] * (c["Hq"] + 2 * c["Hkv"]) * c["d"] <= 2.0e8 and c["B"] * c["T"] <= 32768:
            return c


def _lengths(c):
    """Rows of each sequence before the call: spread over [lo, hi], the first at hi."""
    span = c["hi"] - c["lo"] + 1
    return [c["hi"]] + [c["lo"] + (b * 2654435761 >> 7) % span for b in range(1, c["B"])]


def _counts(c):
    """Rows that each sequence appends: all of T for one token, else spread up to T."""
    T = c["T"]
    return [T] + [T if T == 1 else (b * 2246822519 >> 5) % (T + 1) for b in range(1, c["B"])]


def _cap(c):
    cap = c["hi"] + c["T"]
    return -(-cap // 16) * 16 if not c["page"] else -(-cap // c["page"]) * c["page"]


def _child_counts(n):
    """A draft tree of n nodes: every node has 3 children, from the root on, as long as there are nodes."""
    counts, named = [], 1
    for _ in range(n):
        k = min(3, n - named)
        counts.append(k)
        named += k
    return counts


def _depths(n):
    depth, named = [0], 1
    for i, k in enumerate(_child_counts(n)):
        depth += [depth[i] + 1] * k
    return depth


def work(c):
    if c["op"] == "sample":
        e = 2 if c["type"] == "bf16" else 4
        return dict(bytes=c["rows"] * (c["V"] * e + 5 * 4 + 8), flops=0)
    heads, e = c["Hq"] + 2 * c["Hkv"], 1 if c["type"] == "e4m3" else 2
    if c["op"] == "rope":
        rows = c["B"] * c["T"]
        by = rows * heads * c["d"] * 4 + 4 * c["B"]
    else:
        rows = sum(_counts(c))
        by = rows * c["d"] * (4 * c["Hq"] + 2 * c["Hkv"] * (2 + e)) + 16 * c["B"]
    return dict(bytes=by, flops=rows * (c["Hq"] + c["Hkv"]) * (3 * c["rot"] + (4 * c["d"] if c["norm"] else 0)))


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    def normal(*shape):
        return torch.empty(*shape, device="cuda").normal_(generator=g)

    if c["op"] == "sample":
        _prepare_sample(c, s, uniform, normal)
    else:
        _prepare_rope(c, s, uniform, normal, g)
    if own:
        _prepare_own(c, s)
    return s


def _prepare_rope(c, s, uniform, normal, g):
    B, T, Hq, Hkv, d = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"]
    wide = torch.float16 if c["type"] == "f16" else torch.bfloat16
    # the projection's output holds a token's queries, keys and values side by side
    qkv = (normal(B, T, Hq + 2 * Hkv, d) * (1.0 + uniform(1, 1, Hq + 2 * Hkv, 1))).to(wide)
    s["Q"], s["K"], s["V"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    s["inv_freq"] = (1e6 if c["norm"] else 1e4) ** (-torch.arange(0, c["rot"], 2, device="cuda").float() / c["rot"])
    s["q_norm"] = 1.0 + 0.2 * normal(d) if c["norm"] else None
    s["k_norm"] = 1.0 + 0.2 * normal(d) if c["norm"] else None
    s["Qo"] = torch.zeros(B, T, Hq, d, dtype=wide, device="cuda")
    s["pos"] = (c["far"] * uniform(B)).to(torch.int32)
    if c["op"] == "rope":
        s["Ko"] = torch.zeros(B, T, Hkv, d, dtype=wide, device="cuda")
        s["Vo"] = torch.zeros_like(s["Ko"])
        s["off"] = torch.tensor(_depths(T) if c["tree"] else list(range(T)), dtype=torch.int32, device="cuda")
        return
    s["off"] = torch.arange(T, dtype=torch.int32, device="cuda")
    ps, cap, L = c["page"], _cap(c), _lengths(c)
    s["L"] = torch.tensor(L, dtype=torch.int32, device="cuda")
    s["L0"] = s["L"].clone()
    if c["far"] == 0:
        s["pos"] = None  # a row's position is its place in the cache
    s["counts"] = torch.tensor(_counts(c), dtype=torch.int32, device="cuda")
    s["pt"] = None
    shape = (B, Hkv, cap, d)
    if ps:
        need = [-(-(n + T) // ps) for n in L]
        P = sum(need) + 7
        perm = torch.randperm(P, device="cuda", generator=g).to(torch.int32)
        s["pt"] = torch.full((B, cap // ps), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):  # pages from a shared pool, in no order
            s["pt"][b, :n] = perm[at:at + n]
            at += n
        shape = (P, Hkv, ps, d)
    s["Kc"], s["Vc"] = (normal(*shape).to(TYPES[c["type"]]) for _ in range(2))
    s["k_scale"] = s["v_scale"] = None
    if c["type"] == "e4m3":  # scales as a calibration leaves them: the largest value of a head near 448
        s["k_scale"], s["v_scale"] = (8.0 + uniform(Hkv)) / E4M3_MAX, (8.0 + uniform(Hkv)) / E4M3_MAX


def _prepare_sample(c, s, uniform, normal):
    rows, V = c["rows"], c["V"]
    x = normal(rows, V + c["pad"]) * c["spread"]
    # a model's logits: one token well above the noise, some alternates
    at = (uniform(rows, 8) * V).long().clamp(max=V - 1)
    lift = torch.tensor([6.0] + [3.0] * 7, device="cuda") * c["spread"]
    x.scatter_add_(1, at, lift.expand(rows, 8))
    # a few rows are held to a grammar: half of their tokens are masked
    held = uniform(rows, 1) < 0.1
    x.masked_fill_(held & (uniform(1, V + c["pad"]) < 0.5), -math.inf)
    s["logits"] = x.to(TYPES[c["type"]])
    s["U"] = uniform(rows)
    rule = c["rule"]

    def some(value, off, share):
        return value if rule != "mixed" else torch.where(uniform(rows) < share, value, off)

    s["temperature"] = some(0.3 + uniform(rows), 0.0, 0.95)  # 0: greedy
    s["top_k"] = s["top_p"] = s["min_p"] = None
    if rule in ("top_k", "mixed"):
        s["top_k"] = some(torch.exp(uniform(rows) * math.log(1000.0)), 0.0, 0.5).int()
    if rule in ("top_p", "mixed"):
        s["top_p"] = some(0.5 + 0.49 * uniform(rows), 1.0, 0.7)
    if rule in ("min_p", "mixed"):
        s["min_p"] = some(0.01 + 0.2 * uniform(rows), 0.0, 0.3)
    s["token"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
    s["logprob"] = torch.zeros(rows, device="cuda")


def _prepare_own(c, s):
    import free_speculative_decoding_gb300 as tr
    s["tr"] = tr
    if c["op"] == "sample":
        return
    s["rope"] = tr.Rope(c["d"], s["inv_freq"], pairs=c["pairs"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
    if c["op"] == "rope":
        s["plan"] = tr.Tree(_child_counts(c["T"]), 3) if c["tree"] else None
        return
    s["cache"] = tr.KVCache(s["Kc"], s["Vc"], s["L"], page_table=s["pt"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    s["ws"] = tr.workspace(tr.tr_kv_append_workspace_bytes(s["cache"]))


def _run_own(s):
    tr = s["tr"]
    if s["op"] == "rope":
        tr.tr_qkv_rope(s["Q"], s["K"], s["V"], s["rope"], s["pos"], s["Qo"], s["Ko"], s["Vo"], tree=s["plan"])
    elif s["op"] == "append":
        tr.tr_kv_append_rope(s["Q"], s["K"], s["V"], s["rope"], s["cache"], s["Qo"], s["ws"], pos=s["pos"],
                             count=s["counts"])
    else:
        tr.tr_sample(s["logits"], s["U"], s["token"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                     min_p=s["min_p"], logprob=s["logprob"], V=s["V"])


def _turned(s, x, weight, pos):
    """Rows x [..., H, d] normed and rotated by their positions pos [...], in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    rot = s["rot"]
    angle = pos.double().unsqueeze(-1) * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float().unsqueeze(-2), torch.sin(angle).float().unsqueeze(-2)
    y = x.clone()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if s["pairs"] else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rope(s):
    pos = s["pos"].view(-1, 1) + s["off"]
    s["Qo"].copy_(_turned(s, s["Q"], s["q_norm"], pos))
    s["Ko"].copy_(_turned(s, s["K"], s["k_norm"], pos))
    s["Vo"].copy_(s["V"])


def _raw(x):
    """An 8-bit tensor as bytes, which indexing moves."""
    return x.view(torch.uint8) if x.element_size() == 1 else x


def _plain_append(s):
    B, T, Hkv = s["B"], s["T"], s["Hkv"]
    first = s["L"] if s["pos"] is None else s["pos"]
    b, i = torch.nonzero(s["off"] < s["counts"].view(B, 1), as_tuple=True)
    pos = first[b] + s["off"][i]
    s["Qo"][b, i] = _turned(s, s["Q"][b, i], s["q_norm"], pos).to(s["Qo"].dtype)
    slot = s["L"].long()[b] + i
    ps = s["page"]
    page, at = (b, slot) if s["pt"] is None else (s["pt"][b, slot // ps].long(), slot % ps)
    for r, x, scale in ((_turned(s, s["K"][b, i], s["k_norm"], pos), s["Kc"], s["k_scale"]),
                        (s["V"][b, i].float(), s["Vc"], s["v_scale"])):
        if scale is not None:
            r = (r / scale.view(Hkv, 1)).clamp(-E4M3_MAX, E4M3_MAX)
        _raw(x)[page, :, at] = _raw(r.to(x.dtype))
    s["L"] += s["counts"]


def _plain_sample(s):
    rows, V, T = s["rows"], s["V"], s["temperature"].double().view(-1, 1)
    x = s["logits"][:, :V].float()
    v, order = torch.sort(x, dim=1, descending=True, stable=True)  # equal values: the lower token first
    v = v.double()
    m = v[:, :1]
    w = torch.where(v == m, 1.0, torch.exp((v - m) / T)).masked_fill(v == -math.inf, 0.0)
    keep = (T > 0) | (torch.arange(V, device=x.device) < 1)
    if s["top_k"] is not None:
        k = s["top_k"].view(-1, 1)
        keep = keep & ((k <= 0) | (torch.arange(V, device=x.device) < k))
    w = w * keep
    if s["top_p"] is not None:
        p = s["top_p"].double().view(-1, 1)
        before = torch.cumsum(w, 1) - w
        w = w * ((before < p * w.sum(1, keepdim=True)) | (p >= 1))
    if s["min_p"] is not None:
        low = s["min_p"].double().view(-1, 1)
        w = w * ((low <= 0) | (v >= m + T * torch.log(low)))
    w = torch.zeros_like(w).scatter_(1, order, w)
    mass = torch.cumsum(w, 1)
    total = mass[:, -1:]
    over = (mass > s["U"].double().view(-1, 1) * total) & (w > 0)
    token = torch.where(over, torch.arange(V, device=x.device), V).amin(1, keepdim=True)
    found = token < V
    chosen = w.gather(1, token.clamp(max=V - 1))
    s["token"].copy_(torch.where(found, token, -1).view(rows))
    s["logprob"].copy_(torch.where(found, torch.log(chosen / total), -math.inf).view(rows))


def run(s):
    if s["op"] == "append":
        s["L"].copy_(s["L0"])  # a pass starts where the first one did
    if own:
        _run_own(s)
    elif s["op"] == "rope":
        _plain_rope(s)
    elif s["op"] == "append":
        _plain_append(s)
    else:
        _plain_sample(s)
    if s["op"] == "rope":
        return dict(Q=s["Qo"], K=s["Ko"], V=s["Vo"])
    if s["op"] == "append":
        return dict(Q=s["Qo"], K=s["Kc"], V=s["Vc"], L=s["L"])
    return dict(token=s["token"], logprob=s["logprob"])


def _rotated64(c, s, x, weight, pos):
    """x [n, H, d] of the positions pos [n] in 64 bits: pairs of values as complex numbers, turned."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / c["d"] + EPS) * weight.double()
    rot = c["rot"]
    head, tail = x[..., :rot], x[..., rot:]
    z = head.unflatten(-1, (rot // 2, 2)) if c["pairs"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    angle = (pos.double()[:, None] * s["inv_freq"].double()[None])[:, None]
    z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(angle), angle)
    z = torch.view_as_real(z)
    head = z.flatten(-2) if c["pairs"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat((head, tail), -1)


def _e4m3_of(x, scale):
    """x / scale rounded to the nearest e4m3 value (3 fraction bits, exponents from -6, at most 448), in 64 bits."""
    q = x / scale.double()
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_sample(c, s):
    rows, V = c["rows"], c["V"]
    token = torch.full((rows,), -1, dtype=torch.int32)
    logprob = torch.full((rows,), -math.inf, dtype=torch.float64)
    cpu = {k: None if s[k] is None else s[k].tolist() for k in ("temperature", "top_k", "top_p", "min_p", "U")}
    for r in range(rows):
        x = s["logits"][r, :V].double()
        T, m = cpu["temperature"][r], x.max()
        if T == 0.0:
            token[r], logprob[r] = int((x == m).nonzero()[0]), 0.0
            continue
        ids = torch.nonzero(x > -math.inf).view(-1)
        p = torch.softmax(x[ids] / T, 0)
        rank = torch.argsort(x[ids], descending=True, stable=True)
        if cpu["top_k"] is not None and cpu["top_k"][r] > 0:
            rank = rank[:cpu["top_k"][r]]
        if cpu["top_p"] is not None and cpu["top_p"][r] < 1.0:
            mass = p[rank].cumsum(0)
            enough = torch.nonzero(mass >= cpu["top_p"][r] * mass[-1]).view(-1)
            rank = rank[:int(enough[0]) + 1] if len(enough) else rank
        if cpu["min_p"] is not None and cpu["min_p"][r] > 0.0:
            rank = rank[x[ids[rank]] >= m + T * math.log(cpu["min_p"][r])]
        rank = rank.sort().values
        mass = p[rank].cumsum(0)
        k = min(int((mass <= cpu["U"][r] * mass[-1]).sum()), len(rank) - 1)
        token[r], logprob[r] = int(ids[rank[k]]), float(torch.log(p[rank[k]] / mass[-1]))
    return dict(token=token, logprob=logprob)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "sample":
        return _exact_sample(c, s)
    B, T = c["B"], c["T"]
    if c["op"] == "rope":
        Q, K = torch.empty(s["Qo"].shape, dtype=torch.float64, device="cuda"), torch.empty_like(s["Ko"].double())
        for b in range(B):
            pos = s["pos"][b] + s["off"]
            Q[b], K[b] = _rotated64(c, s, s["Q"][b], s["q_norm"], pos), _rotated64(c, s, s["K"][b], s["k_norm"], pos)
        return dict(Q=Q, K=K, V=s["V"].double())
    Q, L = torch.zeros(s["Qo"].shape, dtype=torch.float64, device="cuda"), s["L"].clone()
    K, V = s["Kc"].double(), s["Vc"].double()
    for b, (n, t) in enumerate(zip(_lengths(c), _counts(c))):
        L[b] = n + t
        pos = s["off"][:t] + (n if s["pos"] is None else s["pos"][b])
        Q[b, :t] = _rotated64(c, s, s["Q"][b, :t], s["q_norm"], pos)
        for new, x, scale in ((_rotated64(c, s, s["K"][b, :t], s["k_norm"], pos), K, s["k_scale"]),
                              (s["V"][b, :t].double(), V, s["v_scale"])):
            r = new.transpose(0, 1)  # [Hkv, t, d]
            if scale is not None:
                r = _e4m3_of(r, scale.view(-1, 1, 1))
            if s["pt"] is None:
                x[b, :, n:n + t] = r
                continue
            ps, at = c["page"], n
            while at < n + t:  # page by page
                k = min(ps - at % ps, n + t - at)
                x[int(s["pt"][b, at // ps]), :, at % ps:at % ps + k] = r[:, at - n:at - n + k]
                at += k
    return dict(Q=Q, K=K, V=V, L=L)
