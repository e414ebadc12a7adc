"""The single-token decode operators and their cases: attention of one new token over a KV cache (tr_decode_attn),
appending rows to that cache (tr_kv_append) and evicting rows from it by accumulated attention weight (tr_kv_evict).

`run` computes them in plain torch operations in 32 bits, or, with `own` set, calls the package's operators."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


def listed():
    return [
        # one sequence at the latency-bound workload's prefix (32 heads): the smallest step a user waits for
        dict(name="decode_1x512_mha", op="decode", type="bf16", B=1, Hkv=32, G=1, d=128, lo=512, hi=512, page=0,
             scores=False),
        # the batched workload's shapes, its cache in pages: 16 sequences with prefixes of 1k to 4k
        dict(name="decode_16x4k_mha_paged", op="decode", type="bf16", B=16, Hkv=32, G=1, d=128, lo=1024, hi=4096,
             page=64, scores=False),
        # the grouped-query workload's shapes, gathering the weights that eviction goes by
        dict(name="decode_8x4k_gqa_scores", op="decode", type="bf16", B=8, Hkv=8, G=4, d=128, lo=4096, hi=4096,
             page=0, scores=True),
        # the long workload: 4 sequences at prefix 32768, the largest read
        dict(name="decode_4x32k_mha", op="decode", type="bf16", B=4, Hkv=32, G=1, d=128, lo=32768, hi=32768, page=0,
             scores=False),
        # a serving batch: 64 requests of any age, 8-bit cache in small pages
        dict(name="decode_64xragged_e4m3", op="decode", type="e4m3", B=64, Hkv=8, G=4, d=128, lo=1, hi=8191, page=16,
             scores=True),
        # a small model: heads of 64, an odd group, fp16, odd lengths
        dict(name="decode_24xodd_f16_d64", op="decode", type="f16", B=24, Hkv=5, G=3, d=64, lo=17, hi=2011, page=32,
             scores=False),
        # one KV head for all query heads (more than one matrix tile of query rows)
        dict(name="decode_4x16k_mqa", op="decode", type="bf16", B=4, Hkv=1, G=40, d=128, lo=9001, hi=16001, page=128,
             scores=True),
        # the new token of each sequence of the batched workload
        dict(name="append_16x1", op="append", type="bf16", B=16, Hkv=32, d=128, T=1, lo=1024, hi=4096, page=64),
        # prompts of up to 4096 tokens taken into an 8-bit cache
        dict(name="append_8x4k_e4m3", op="append", type="e4m3", B=8, Hkv=8, d=128, T=4096, lo=0, hi=300, page=16),
        # the batched workload's caches cut down to 1024 rows each, dense
        dict(name="evict_16x4k_to_1k", op="evict", type="bf16", B=16, Hkv=32, d=128, lo=2048, hi=4096, page=0,
             budget=1024, recent=256),
        # one very long sequence in pages cut to a quarter
        dict(name="evict_1x128k_to_32k", op="evict", type="bf16", B=1, Hkv=8, d=128, lo=131072, hi=131072, page=64,
             budget=32768, recent=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    while True:
        op = rng.choice(("decode", "decode", "decode", "append", "evict"))
        c = dict(op=op, type=rng.choice(("bf16", "bf16", "f16", "e4m3")), B=_log(rng, 1, 64),
                 Hkv=rng.choice((1, 2, 4, 5, 8, 16, 32)), d=rng.choice((64, 128, 128)),
                 page=rng.choice((0, 16, 32, 64, 128, 256)))
        if op == "decode":
            c["G"] = rng.choice((1, 1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 40))
            c["hi"] = _log(rng, 1, 32768)
            c["lo"] = rng.choice((c["hi"], max(1, c["hi"] // 4), 1, 0))
            c["scores"] = rng.random() < 0.4
        elif op == "append":
            c["T"] = _log(rng, 1, 4096)
            c["hi"] = _log(rng, 1, 8192)
            c["lo"] = rng.choice((c["hi"], 0))
        else:
            c["hi"] = _log(rng, 64, 131072)
            c["lo"] = max(0, int(c["hi"] * rng.choice((1.0, 0.5, 0.0))))
            c["budget"] = max(2, int(c["hi"] * rng.uniform(0.1, 0.9)))
            c["recent"] = int(c["budget"] * rng.uniform(0.0, 0.6))
        c["page"] = min(c["page"], 256)
        if 2e5 <= work(c)["bytes"] <= 2e9:
            return c


def _lengths(c):
    """Rows of each sequence before the call: spread over [lo, hi], the first at hi."""
    span = c["hi"] - c["lo"] + 1
    return [c["hi"]] + [c["lo"] + (b * 2654435761 >> 7) % span for b in range(1, c["B"])]


def _counts(c):
    """Rows that each sequence appends: all of T for one token, else spread up to T."""
    T = c["T"]
    return [T] + [T if T == 1 else (b * 2246822519 >> 5) % (T + 1) for b in range(1, c["B"])]


def _esize(c):
    return 1 if c["type"] == "e4m3" else 2


def _cap(c):
    cap = c["hi"] + c.get("T", 0)
    return -(-cap // 16) * 16 if not c["page"] else -(-cap // c["page"]) * c["page"]


def work(c):
    L, row = _lengths(c), c["Hkv"] * c["d"] * _esize(c)
    if c["op"] == "decode":
        rows, Hq = sum(L), c["Hkv"] * c["G"]
        by = 2 * rows * row + c["B"] * Hq * (c["d"] * 2 + c["d"] * 4 + 4) + 4 * c["B"]
        by += 8 * rows * c["Hkv"] if c["scores"] else 0
        return dict(bytes=by, flops=4 * rows * Hq * c["d"])
    if c["op"] == "append":
        rows = sum(_counts(c))
        return dict(bytes=2 * rows * (row + c["Hkv"] * c["d"] * 2) + 4 * rows * c["Hkv"] + 8 * c["B"], flops=0)
    over = [n for n in L if n > c["budget"]]
    # every score is read, every kept row and score is read and written
    by = 4 * c["Hkv"] * sum(over) + len(over) * c["budget"] * (4 * row + 4 * c["Hkv"]) + 8 * c["B"]
    return dict(bytes=by, flops=0)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, wide = TYPES[c["type"]], torch.float16 if c["type"] == "f16" else torch.bfloat16
    B, Hkv, d, ps, cap = c["B"], c["Hkv"], c["d"], c["page"], _cap(c)
    L = _lengths(c)

    def rows(shape, scale=None):
        x = torch.empty(shape, dtype=wide, device="cuda").normal_(generator=g)
        return x if scale is None else (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(dt)

    s = dict(c)
    s["k_scale"] = s["v_scale"] = ks = vs = None
    if c["type"] == "e4m3":  # scales as a calibration leaves them: the largest value of a head near 448
        s["k_scale"] = (4.5 + torch.rand(Hkv, device="cuda", generator=g)) / E4M3_MAX
        s["v_scale"] = (4.5 + torch.rand(Hkv, device="cuda", generator=g)) / E4M3_MAX
        ks, vs = s["k_scale"].view(Hkv, 1, 1), s["v_scale"].view(Hkv, 1, 1)
    s["pt"] = None
    if ps:
        mp = cap // ps
        need = [-(-(n + (c["T"] if c["op"] == "append" else 0)) // ps) for n in L]
        P = sum(need) + 7
        perm = torch.randperm(P, device="cuda", generator=g).to(torch.int32)
        pt = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):  # pages from a shared pool, in no order
            pt[b, :n] = perm[at:at + n]
            at += n
        s["pt"] = pt
        s["K"], s["V"] = rows((P, Hkv, ps, d), ks), rows((P, Hkv, ps, d), vs)
    else:
        s["K"], s["V"] = rows((B, Hkv, cap, d), ks), rows((B, Hkv, cap, d), vs)
    s["L"] = torch.tensor(L, dtype=torch.int32, device="cuda")
    s["L0"] = s["L"].clone()
    s["scores"] = s["counts"] = None
    s["cap"], s["Lmax"] = cap, max(L)
    s["scale"] = d ** -0.5
    if c["op"] == "decode":
        Hq = Hkv * c["G"]
        # queries that give logits with a spread of about 2: some keys carry most of the weight
        s["Q"] = (2.0 * torch.empty(B, Hq, d, device="cuda").normal_(generator=g)).to(wide)
        s["O"] = torch.empty(B, Hq, d, dtype=torch.float32, device="cuda")
        s["lse"] = torch.empty(B, Hq, dtype=torch.float32, device="cuda")
        if c["scores"]:
            s["scores"] = torch.rand(B, Hkv, cap, device="cuda", generator=g)
    elif c["op"] == "append":
        s["Kn"], s["Vn"] = rows((B, c["T"], Hkv, d)), rows((B, c["T"], Hkv, d))
        s["counts"] = torch.tensor(_counts(c), dtype=torch.int32, device="cuda")
        s["scores"] = torch.rand(B, Hkv, cap, device="cuda", generator=g)
    else:
        # accumulated weights have a long tail; rows that no query has looked at yet have none
        sc = torch.empty(B, Hkv, cap, device="cuda").normal_(generator=g).mul_(1.5).exp_()
        s["scores0"] = sc * (torch.rand(B, Hkv, cap, device="cuda", generator=g) > 0.05)
        s["scores"] = s["scores0"].clone()
    if own:
        import free_speculative_decoding_gb300 as tr
        s["tr"] = tr
        s["cache"] = tr.KVCache(s["K"], s["V"], s["L"], page_table=s["pt"], scores=s["scores"],
                                k_scale=s["k_scale"], v_scale=s["v_scale"])
        if c["op"] == "decode":
            nb = tr.tr_decode_attn_workspace_bytes(s["cache"], Hkv * c["G"], accumulate=c["scores"])
        elif c["op"] == "append":
            nb = tr.tr_kv_append_workspace_bytes(s["cache"])
        else:
            nb = tr.tr_kv_evict_workspace_bytes(s["cache"], c["budget"])
        s["ws"] = tr.workspace(nb)
    return s


def _run_own(s):
    tr, cache = s["tr"], s["cache"]
    if s["op"] == "decode":
        tr.tr_decode_attn(s["Q"], cache, s["O"], s["scale"], s["ws"], lse=s["lse"], accumulate=s["scores"] is not None)
    elif s["op"] == "append":
        tr.tr_kv_append(s["Kn"], s["Vn"], cache, s["ws"], count=s["counts"])
    else:
        tr.tr_kv_evict(cache, s["budget"], s["recent"], s["ws"])


def _at(s, slots):
    """Index of the rows `slots` [B, Hkv, n] of a cache tensor."""
    B, Hkv = slots.shape[:2]
    h = torch.arange(Hkv, device=slots.device).view(1, Hkv, 1)
    if s["pt"] is None:
        return torch.arange(B, device=slots.device).view(B, 1, 1), h, slots
    page = s["pt"].long().gather(1, (slots // s["page"]).reshape(B, -1)).view(slots.shape)
    return page, h, slots % s["page"]


def _raw(x):
    """An 8-bit tensor as bytes, which indexing moves."""
    return x.view(torch.uint8) if x.element_size() == 1 else x


def _rows32(s, x, scale):
    """The first Lmax rows of every sequence of a cache tensor in 32 bits, [B, Hkv, Lmax, d]."""
    n = s["Lmax"]
    if s["pt"] is None:
        r = x[:, :, :n]
    else:
        pages = s["pt"][:, :-(-n // s["page"])].clamp(min=0).long()
        r = _raw(x)[pages].view(x.dtype)  # [B, pages, Hkv, page, d]
        r = r.transpose(1, 2).reshape(s["B"], s["Hkv"], -1, s["d"])[:, :, :n]
    r = r.float()
    return r if scale is None else r * scale.view(1, -1, 1, 1)


def _plain_decode(s):
    B, Hkv, G, d, n = s["B"], s["Hkv"], s["G"], s["d"], s["Lmax"]
    seen = (torch.arange(n, device="cuda") < s["L"].view(B, 1)).view(B, 1, 1, n)
    q = s["Q"].float().view(B, Hkv, G, d) * s["scale"]
    x = q @ _rows32(s, s["K"], s["k_scale"]).transpose(2, 3)
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(3, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - m)
    l = p.sum(3, keepdim=True)
    v = _rows32(s, s["V"], s["v_scale"]).masked_fill(~seen.view(B, 1, n, 1), 0.0)
    w = torch.where(l > 0, p / l, 0.0)
    if s["scores"] is not None:
        s["scores"][:, :, :n] += w.sum(2)
    return (w @ v).view(B, Hkv * G, d), (m + torch.log(l)).view(B, Hkv * G)


def _plain_append(s):
    B, T, Hkv, d = s["Kn"].shape
    i = torch.arange(T, device="cuda")
    b, i = torch.nonzero(i < s["counts"].view(B, 1), as_tuple=True)
    slot = s["L"].long()[b] + i
    page, off = (b, slot) if s["pt"] is None else (s["pt"][b, slot // s["page"]].long(), slot % s["page"])
    for new, x, scale in ((s["Kn"], s["K"], s["k_scale"]), (s["Vn"], s["V"], s["v_scale"])):
        r = new[b, i]
        if scale is not None:
            r = (r.float() / scale.view(Hkv, 1)).clamp(-E4M3_MAX, E4M3_MAX).to(x.dtype)
        _raw(x)[page, :, off] = _raw(r)
    s["scores"][b, :, slot] = 0.0
    s["L"] += s["counts"]


def _plain_evict(s):
    n, k, B, Hkv = s["Lmax"], s["budget"], s["B"], s["Hkv"]
    if n > k:
        slot = torch.arange(n, device="cuda")
        L = s["L"].view(B, 1, 1).long()
        key = s["scores"][:, :, :n].masked_fill(slot >= L - s["recent"], math.inf).masked_fill(slot >= L, -math.inf)
        order = torch.sort(key, dim=2, descending=True, stable=True).indices[:, :, :k]
        keep = torch.where(L > k, order.sort(dim=2).values, slot[:k])
        # a sequence within the budget keeps its rows where they are (and has no pages behind them)
        b, h, r = torch.nonzero((L > k).expand(B, Hkv, k), as_tuple=True)
        src = keep[b, h, r]
        if s["pt"] is None:
            frm, to = (b, h, src), (b, h, r)
        else:
            frm = (s["pt"][b, src // s["page"]].long(), h, src % s["page"])
            to = (s["pt"][b, r // s["page"]].long(), h, r % s["page"])
        _raw(s["K"])[to] = _raw(s["K"])[frm]
        _raw(s["V"])[to] = _raw(s["V"])[frm]
        s["scores"][b, h, r] = s["scores"][b, h, src]
    s["L"].clamp_(max=k)


def run(s):
    # a pass starts where the first one did: lengths (and the scores that an eviction moves) are put back
    if s["op"] != "decode":
        s["L"].copy_(s["L0"])
    if s["op"] == "evict":
        s["scores"].copy_(s["scores0"])
    if s["op"] == "decode":
        if own:
            _run_own(s)
            O, lse = s["O"], s["lse"]
        else:
            O, lse = _plain_decode(s)
        return dict(O=O, lse=lse) if s["scores"] is None else dict(O=O, lse=lse, scores=s["scores"])
    if own:
        _run_own(s)
    elif s["op"] == "append":
        _plain_append(s)
    else:
        _plain_evict(s)
    return dict(K=s["K"], V=s["V"], scores=s["scores"], L=s["L"])


def _sequence(s, x, b, n):
    """Sequence b's first n rows in 64 bits, [Hkv, n, d]."""
    if s["pt"] is None:
        return x[b, :, :n].double()
    if n == 0:
        return x.new_zeros((s["Hkv"], 0, s["d"]), dtype=torch.float64)
    pages = [x[int(p)].double() for p in s["pt"][b, :-(-n // s["page"])].tolist()]
    return torch.cat(pages, 1)[:, :n]


def _e4m3_of(x, scale):
    """x / scale rounded to the nearest e4m3 value (3 fraction bits, exponents from -6, at most 448), in 64 bits."""
    q = x.double() / scale.double()
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(c, seed):
    s = prepare(c, seed)
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "decode":
        G = c["G"]
        O = torch.zeros(B, Hkv * G, d, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hkv * G), -math.inf, dtype=torch.float64, device="cuda")
        sc = None if s["scores"] is None else s["scores"].double()
        for b, n in enumerate(_lengths(c)):
            if n == 0:
                continue
            k, v = _sequence(s, s["K"], b, n), _sequence(s, s["V"], b, n)
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"].double().view(-1, 1, 1), v * s["v_scale"].double().view(-1, 1, 1)
            for h in range(Hkv):
                z = (k[h] @ s["Q"][b, h * G:(h + 1) * G].double().T) * d ** -0.5  # [n, G]
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(z, 0)
                w = torch.softmax(z, 0)
                O[b, h * G:(h + 1) * G] = w.T @ v[h]
                if sc is not None:
                    sc[b, h, :n] += w.sum(1)
        return dict(O=O, lse=lse) if sc is None else dict(O=O, lse=lse, scores=sc)
    K, V, sc = s["K"], s["V"], s["scores"].clone()
    L = s["L"].clone()
    if c["op"] == "append":
        K, V = K.double(), V.double()
        for b, (n, t) in enumerate(zip(_lengths(c), _counts(c))):
            L[b] = n + t
            sc[b, :, n:n + t] = 0
            for new, x, scale in ((s["Kn"], K, s["k_scale"]), (s["Vn"], V, s["v_scale"])):
                r = new[b, :t].transpose(0, 1)  # [Hkv, t, d]
                r = r.double() if scale is None else _e4m3_of(r, scale.view(-1, 1, 1))
                if s["pt"] is None:
                    x[b, :, n:n + t] = r
                    continue
                ps, at = c["page"], n
                while at < n + t:  # page by page
                    m = min(ps - at % ps, n + t - at)
                    x[int(s["pt"][b, at // ps]), :, at % ps:at % ps + m] = r[:, at - n:at - n + m]
                    at += m
        return dict(K=K, V=V, scores=sc, L=L)
    if c["type"] == "e4m3":
        K, V = K.float(), V.float()
    for b, n in enumerate(_lengths(c)):
        k, r = c["budget"], c["recent"]
        if n <= k:
            continue
        L[b] = k
        if s["pt"] is not None:
            used = s["pt"][b, :-(-n // c["page"])].long()
        for h in range(Hkv):
            kept = torch.ones(n, dtype=torch.bool, device="cuda")
            old = s["scores"][b, h, :n - r].double()
            if k - r < n - r:
                if k > r:
                    edge = torch.kthvalue(-old, k - r).values.neg()
                    above, tie = old > edge, old == edge
                    kept[:n - r] = above | (tie & (tie.long().cumsum(0) <= k - r - above.sum()))
                else:
                    kept[:n - r] = False
            if s["pt"] is None:
                for x in (K, V):
                    x[b, h, :k] = x[b, h, :n][kept]
            else:
                ps = c["page"]
                for x in (K, V):
                    rows = x[used, h].reshape(-1, d)
                    rows = torch.cat((rows[:n][kept], rows[k:]))
                    x[used, h] = rows.view(-1, ps, d)
            sc[b, h, :k] = sc[b, h, :n][kept]
    return dict(K=K, V=V, scores=sc, L=L)
