"""Measured cases of the operators of a batch's decode step on a paged cache: appending with the norms of queries
and keys, attention over a prefix that requests share (and the weights it gives to what they do not), and eviction
by accumulated weight.

`run` computes them in plain torch operations, or (own = True) through the package's own calls.  A cache is
[pages][page tokens][record] bf16 behind an int32 page table [requests][pages of a request]; a record is per KV
head [K | V] ("gqa") or one latent whose tail is the rotated part and whose first dim_v values are V ("latent").
"""
import math
import random

import torch

own = False

GQA = {"layout": "gqa", "q_heads": 32, "kv_heads": 8, "dim_qk": 128, "dim_v": 128}
LATENT = {"layout": "latent", "q_heads": 64, "kv_heads": 1, "dim_qk": 576, "dim_v": 512}
EPS = 1e-6


def listed():
    return [
        # a decode step of batch 16: one token a request, norms of queries and keys, latency alone counts
        dict(GQA, name="norm_step_b16", op="norm", requests=16, tokens=16, first=131000, page=64, rotary=128,
             interleaved=False, axes=1, weight="bf16", per_head=False),
        # a prefill chunk of four ragged prompts far into long contexts
        dict(GQA, name="norm_chunk", op="norm", requests=4, tokens=16384, first=1000000, page=64, rotary=128,
             interleaved=False, axes=1, weight="bf16", per_head=False),
        # images and video among text: three axes of positions, half of each head rotated, weights for each head
        dict(GQA, name="norm_axes_chunk", op="norm", q_heads=40, requests=3, tokens=6001, first=5000, page=16, rotary=64,
             interleaved=True, axes=3, weight="fp32", per_head=True),
        # shared-latent prefill chunk: the latent's norm, its rotary tail and the queries' rotary part
        dict(LATENT, name="norm_latent_chunk", op="norm", requests=5, tokens=8191, first=777, page=64, rotary=64,
             interleaved=True, axes=1, weight="bf16", per_head=False),
        # two short chats with one system prompt: latency alone counts
        dict(GQA, name="prefix_pair_short", op="prefix", requests=2, groups=1, loose=0, prefix=700, own=300, page=64,
             weigh="", decay=1.0),
        # the benchmark's batch of 16 over one document, some thousand own tokens each
        dict(GQA, name="prefix_b16", op="prefix", requests=16, groups=1, loose=0, prefix=32768, own=2048, page=64,
             weigh="", decay=1.0),
        # a large batch of short questions about one long document
        dict(GQA, name="prefix_long_b64", op="prefix", requests=64, groups=1, loose=0, prefix=131072, own=1000, page=64,
             weigh="", decay=1.0),
        # three system prompts of different lengths, some requests with none, small odd heads
        dict(GQA, name="prefix_groups_b48", op="prefix", q_heads=28, kv_heads=4, dim_qk=64, dim_v=64, requests=48, groups=3,
             loose=5, prefix=12001, own=1500, page=16, weigh="", decay=1.0),
        # the shared-latent batch of the benchmark over one document
        dict(LATENT, name="prefix_latent_b8", op="prefix", requests=8, groups=1, loose=0, prefix=32768, own=600, page=64,
             weigh="", decay=1.0),
        # a decode step that keeps account of what is attended, for each KV head, without a shared prefix
        dict(GQA, name="weigh_b16", op="prefix", requests=16, groups=0, loose=16, prefix=0, own=8192, page=64,
             weigh="heads", decay=1.0),
        # one request a token over its budget
        dict(GQA, name="evict_one", op="evict", requests=1, context=2049, keep=2048, first=4, recent=64, page=64, lists="one"),
        # a batch cut from 8192 to the benchmark's 4096 entries, each KV head its own
        dict(GQA, name="evict_b16", op="evict", requests=16, context=8192, keep=4096, first=16, recent=512, page=64,
             lists="heads"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "prefix", "prefix", "prefix", "evict", "evict"])
    shape = dict(rng.choice([GQA, GQA, LATENT]))
    latent = shape["layout"] == "latent"
    if not latent:
        shape["kv_heads"] = rng.choice([2, 4, 8])
        shape["q_heads"] = shape["kv_heads"] * rng.choice([1, 2, 4, 5, 7, 8])
        shape["dim_qk"] = shape["dim_v"] = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm":
        return dict(shape, op=op, requests=_spread(rng, 1, 64), tokens=_spread(rng, 1, 8192), first=_spread(rng, 1, 1 << 20),
                    page=page, rotary=64 if latent else rng.choice([32, 64, shape["dim_qk"]]), interleaved=rng.random() < 0.5,
                    axes=rng.choice([1, 1, 2, 3]), weight=rng.choice(["bf16", "fp32"]),
                    per_head=not latent and rng.random() < 0.3)
    if op == "prefix":
        weigh = rng.choice(["", "", "one", "heads"])
        n = _spread(rng, 1, 16 if latent or weigh else 64)
        groups = rng.randint(0, min(3, n))
        own = _spread(rng, 1, 4096 if n <= 16 else 1024)
        return dict(shape, op=op, requests=n, groups=groups, loose=n if groups == 0 else rng.choice([0, 0, (n - groups) // 3]),
                    prefix=_spread(rng, 1, 16384 if latent else 65536) if groups else 0, own=own, page=page, weigh=weigh,
                    decay=rng.choice([1.0, 0.95]) if weigh else 1.0)
    context = _spread(rng, 2, 16384)
    keep = max(1, int(context * rng.uniform(0.1, 0.99)))
    first = rng.choice([0, min(4, keep // 4), keep // 4])
    return dict(shape, op=op, requests=_spread(rng, 1, max(1, min(32, 131072 // context))), context=context, keep=keep,
                first=first, recent=rng.randint(0, keep - first), page=page, lists=rng.choice(["one", "heads"]))


# ---- sizes that go by the case alone -----------------------------------------------------------


def _record(case):
    if case["layout"] == "latent":
        return case["dim_qk"]
    return case["kv_heads"] * (case["dim_qk"] + case["dim_v"])


def _ragged(n, top):
    """n lengths from an eighth of `top` to it, all different where there is room."""
    if n == 1:
        return [top]
    return [max(1, top // 8 + (top - top // 8) * r // (n - 1) - (r * 5) % 7 * (r < n - 1)) for r in range(n)]


def _counts(case):
    """Tokens each request appends: a ragged split (some may append nothing)."""
    n, total = case["requests"], case["tokens"]
    cuts = [total * (r + (r % 3) * (0 < r)) // (n + 2) for r in range(n)] + [total]
    cuts = sorted(min(c, total) for c in cuts) if total > n else [min(r, total) for r in range(n + 1)]
    cuts[0], cuts[-1] = 0, total
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _groups(case):
    """Bounds of the groups among the requests (those behind the last are in none), and their prefixes' lengths."""
    n, g = case["requests"] - case["loose"], case["groups"]
    if g == 0:
        return [0], []
    each = g * (g + 1) // 2  # sizes as 1 : 2 : 3
    cu = [min(n - (g - i), max(i, n * (i * (i + 1) // 2) // each)) for i in range(g)] + [n]
    return cu, [max(1, case["prefix"] * (i + 1) // g - 3 * (g - 1 - i)) for i in range(g)]


def _shared(case):
    """For each request: the first of its group (itself without one), and the positions it shares."""
    cu, prefix = _groups(case)
    lead, pre = list(range(case["requests"])), [0] * case["requests"]
    for g, p in enumerate(prefix):
        for r in range(cu[g], cu[g + 1]):
            lead[r], pre[r] = cu[g], p
    return lead, pre


def _lists(case, key):
    return {"": 0, "one": 1, "heads": case["kv_heads"]}[case[key]]


def _contexts(case):
    """Lengths of the requests of an eviction: some may be within the budget already."""
    return _ragged(case["requests"], case["context"])


def work(case):
    rec, n, hq = 2 * _record(case), case["requests"], case["q_heads"]
    if case["op"] == "norm":
        latent = case["layout"] == "latent"
        width = case["rotary"] if latent else case["dim_qk"]
        values = _record(case) // (1 if latent else 2) + (0 if latent else hq * width)  # normed
        bytes_ = case["tokens"] * (2 * rec + 4 * hq * width + 8 * case["axes"])
        pairs = case["rotary"] // 2 * (case["kv_heads"] + hq)
        return {"bytes": bytes_, "flops": case["tokens"] * (4 * values + 6 * pairs)}
    if case["op"] == "prefix":
        cu, prefix = _groups(case)
        owned = _ragged(n, case["own"])
        entries = sum(prefix) + sum(owned)
        rows = sum(p * (b - a) for p, a, b in zip(prefix, cu, cu[1:])) + sum(owned)  # (request, entry) pairs
        lists = _lists(case, "weigh")
        return {"bytes": entries * rec + 2 * n * hq * (case["dim_qk"] + case["dim_v"]) + 8 * lists * sum(owned),
                "flops": 2 * rows * hq * (case["dim_qk"] + case["dim_v"])}
    lists = _lists(case, "lists")
    moved = sum(case["keep"] - case["first"] for c in _contexts(case) if c > case["keep"])
    return {"bytes": 8 * lists * sum(_contexts(case)) + 2 * moved * rec, "flops": 0}


# ---- inputs ------------------------------------------------------------------------------------


def _config(case):
    from hierarchical_kv_cache_02_gb300 import LAYOUT_GQA, LAYOUT_MLA, HsConfig

    return HsConfig(num_requests=case["requests"], num_layers=1, capacity=1,
                    layout=LAYOUT_MLA if case["layout"] == "latent" else LAYOUT_GQA, num_q_heads=case["q_heads"],
                    num_kv_heads=case["kv_heads"], head_dim_qk=case["dim_qk"], head_dim_v=case["dim_v"], top_k=1,
                    buffer_slots=1)


def _cache(case, most, g):
    """Random pages in a random order, with room for `most` positions a request."""
    n, page = case["requests"], case["page"]
    each = -(-most // page)
    pages = torch.randn((n * each, page, _record(case)), generator=g, device="cuda", dtype=torch.bfloat16)
    table = torch.randperm(n * each, generator=g, device="cuda").to(torch.int32).view(n, each)
    return pages, table


def _prepare_norm(s, case, g):
    n, hq, hk, dq, total = (case[x] for x in ("requests", "q_heads", "kv_heads", "dim_qk", "tokens"))
    latent = case["layout"] == "latent"
    counts = _counts(case)
    s["pages"], s["table"] = _cache(case, max(counts) + case["first"] % 512, g)
    s["cu"] = torch.tensor([sum(counts[:r]) for r in range(n + 1)], dtype=torch.int32, device="cuda")
    # the cache holds the last `first` % 512 positions and what comes; angles count from `first`
    s["start"] = torch.full((n,), case["first"] % 512, dtype=torch.int64, device="cuda")
    at = torch.cat([torch.arange(c, device="cuda") for c in counts]) + case["first"]
    if case["axes"] > 1:
        # time stands still in an image while rows and columns go on
        i = torch.arange(total, device="cuda")
        at = torch.stack([at // 64 * 64, at // 64 * 64 + i % 64 // 8, at // 64 * 64 + i % 8][: case["axes"]], dim=1)
    s["at"] = at.contiguous()
    # keys, values and queries as views of one projection, as a model has them
    kw, vw = hk * dq, 0 if latent else hk * case["dim_v"]
    width = case["rotary"] if latent else dq
    flat = torch.randn((total, hq * width + kw + vw), generator=g, device="cuda")
    flat *= torch.rand((total, 1), generator=g, device="cuda") * 4 + 0.25  # tokens of different norms
    flat = flat.to(torch.bfloat16)
    s["q"] = flat[:, : hq * width].unflatten(1, (hq, width))
    s["q_out"] = torch.empty((total, hq, width), dtype=torch.bfloat16, device="cuda")
    s["k"] = flat[:, hq * width : hq * width + kw].unflatten(1, (hk, dq))
    if vw:
        s["v"] = flat[:, hq * width + kw :].unflatten(1, (hk, case["dim_v"]))
    kind = torch.bfloat16 if case["weight"] == "bf16" else torch.float32

    def weight(heads, dim):
        w = 1.0 + 0.3 * torch.randn((heads, dim) if case["per_head"] else (dim,), generator=g, device="cuda")
        return w.to(kind)

    s["k_weight"] = weight(hk, case["dim_v"] if latent else dq)
    if not latent:
        s["q_weight"] = weight(hq, dq)
    half = case["rotary"] // 2
    s["freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    s["freq_gpu"] = s["freq"].cuda()
    s["axis"] = [j % case["axes"] for j in range(half)]
    s["axis_gpu"] = torch.tensor(s["axis"], device="cuda")


def _prepare_prefix(s, case, g):
    n, hq, dq, page = case["requests"], case["q_heads"], case["dim_qk"], case["page"]
    lead, pre = _shared(case)
    owned = _ragged(n, case["own"])
    cu, prefix = _groups(case)
    # whole pages of a prefix are in the tables of all its requests; a request has its own from there on
    each = max(-(-(p + o) // page) for p, o in zip(pre, owned))
    have = [p // page if lead[r] != r else 0 for r, p in enumerate(pre)]
    need = [-(-(p + o) // page) - h for p, o, h in zip(pre, owned, have)]
    s["pages"] = torch.randn((sum(need), page, _record(case)), generator=g, device="cuda", dtype=torch.bfloat16)
    order = torch.randperm(sum(need), generator=g, device="cuda").tolist()
    table = []
    for r in range(n):
        mine = (table[lead[r]][: have[r]] if have[r] else []) + [order.pop() for _ in range(need[r])]
        table.append(mine + [-1] * (each - len(mine)))  # never read: behind a request's length
    s["table"] = torch.tensor(table, dtype=torch.int32, device="cuda").view(n, each)
    s["lens"] = torch.tensor([p + o for p, o in zip(pre, owned)], dtype=torch.int64, device="cuda")
    s["groups"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["prefix"] = torch.tensor(prefix, dtype=torch.int64, device="cuda")
    s["pre"] = torch.tensor(pre, dtype=torch.int64, device="cuda")
    # heads from flat to peaked softmaxes
    sharp = torch.linspace(0.5, 3.0, hq, device="cuda").view(1, hq, 1)
    s["q"] = (torch.randn((n, hq, dq), generator=g, device="cuda") * sharp).to(torch.bfloat16)
    s["out"] = torch.zeros((n, hq, case["dim_v"]), dtype=torch.bfloat16, device="cuda")
    if case["weigh"]:
        s["weights"] = torch.rand((n, _lists(case, "weigh"), each * page), generator=g, device="cuda")


def _prepare_evict(s, case, g):
    n = case["requests"]
    s["pages"], s["table"] = _cache(case, case["context"], g)
    s["lens"] = torch.tensor(_contexts(case), dtype=torch.int64, device="cuda")
    # sums of attention weights: a few entries have most, many next to nothing, and some none at all
    shape = (n, _lists(case, "lists"), s["table"].shape[1] * case["page"])
    w = torch.exp(2.0 * torch.randn(shape, generator=g, device="cuda"))
    s["weights"] = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.1, 0.0, w)
    s["weights_out"] = torch.zeros(shape, device="cuda")
    s["lens_out"] = torch.zeros_like(s["lens"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    s = {"case": case}
    {"norm": _prepare_norm, "prefix": _prepare_prefix, "evict": _prepare_evict}[case["op"]](s, case, g)
    if own:
        from hierarchical_kv_cache_02_gb300 import PagedKV, RopeTable

        s["kv"] = PagedKV(_config(case), s["pages"], s["table"])
        if case["op"] == "norm":
            s["rope"] = RopeTable(case["rotary"], inv_freq=s["freq"].tolist(), interleaved=case["interleaved"],
                                  axes=s["axis"] if case["axes"] > 1 else None)
    return s


# ---- plain forms -------------------------------------------------------------------------------


def _rows_of(s, positions, requests=None):
    """Flat row of each position [requests][n] in the cache seen as [rows][record]."""
    page = s["case"]["page"]
    table = s["table"].long() if requests is None else s["table"][requests].long()
    return table.gather(1, positions // page) * page + positions % page


def _normed(x, weight):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * weight.float()


def _turned(x, cos, sin, lo, interleaved):
    """x [tokens][heads][dims] in 32 bits with the dims [lo, lo + 2 pairs) rotated."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    part, to = x[..., lo : lo + 2 * half], y[..., lo : lo + 2 * half]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        to[..., 0::2], to[..., 1::2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = part[..., :half], part[..., half:]
        to[..., :half], to[..., half:] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_norm(s):
    case = s["case"]
    t = torch.arange(case["tokens"], device="cuda")
    req = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    at = s["start"][req] + t - s["cu"][req]
    turned_at = s["at"][:, s["axis_gpu"]] if case["axes"] > 1 else s["at"][:, None]
    angle = turned_at.double() * s["freq_gpu"]  # 64 bits: far positions turn many times
    cos, sin = angle.cos().float(), angle.sin().float()
    if case["layout"] == "latent":
        dv = case["dim_v"]
        rec = torch.cat([_normed(s["k"][..., :dv], s["k_weight"]), s["k"][..., dv:].float()], dim=-1)
        rec = _turned(rec, cos, sin, dv, case["interleaved"]).to(torch.bfloat16)
        q = s["q"].float()
    else:
        rec = _turned(_normed(s["k"], s["k_weight"]), cos, sin, 0, case["interleaved"]).to(torch.bfloat16)
        rec = torch.cat([rec, s["v"]], dim=2)
        q = _normed(s["q"], s["q_weight"])
    page = case["page"]
    row = s["table"][req, at // page].long() * page + at % page
    s["pages"].view(-1, _record(case))[row] = rec.reshape(case["tokens"], -1)
    s["q_out"].copy_(_turned(q, cos, sin, 0, case["interleaved"]))
    return [s["pages"], s["q_out"]]


def _keys_values(case, rows):
    """rows [...][entries][record] in 32 bits as keys and values [...][kv heads][entries][dims]."""
    dq, dv = case["dim_qk"], case["dim_v"]
    if case["layout"] == "latent":
        k = rows.float().unsqueeze(-3)
        return k, k[..., :dv]
    rows = rows.unflatten(-1, (case["kv_heads"], dq + dv)).transpose(-2, -3)
    return rows[..., :dq].float(), rows[..., dq:].float()


def _part(q, k, v, seen=None):
    """Unnormalised attention: the sum of weights times values, the largest score and the sum of weights."""
    a = q @ k.transpose(-1, -2)
    a *= 1.0 / math.sqrt(q.shape[-1])
    if seen is not None:
        a.masked_fill_(~seen, -math.inf)
    scores = a.clone() if seen is not None else None
    top = a.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    a.sub_(top).exp_()
    return a @ v, top, a.sum(dim=-1, keepdim=True), scores


def _plain_prefix(s):
    case = s["case"]
    n, hq, hk, dq, dv = (case[x] for x in ("requests", "q_heads", "kv_heads", "dim_qk", "dim_v"))
    g = hq // hk
    flat = s["pages"].view(-1, _record(case))
    q = s["q"].float().view(n, hk, g, dq)
    # what each request has for itself, padded to the longest
    i = torch.arange(case["own"], device="cuda")
    at = s["pre"][:, None] + i
    seen = at < s["lens"][:, None]
    at = torch.where(seen, at, s["pre"][:, None])
    k, v = _keys_values(case, flat[_rows_of(s, at)])
    o, top, total, scores = _part(q, k, v, seen[:, None, None, :])
    cu, prefix = _groups(case)
    for a, b, p in zip(cu, cu[1:], prefix):  # a product for each shared prefix, all its requests' rows at once
        k, v = _keys_values(case, flat[_rows_of(s, torch.arange(p, device="cuda")[None], slice(a, a + 1))[0]])
        rows = q[a:b].transpose(0, 1).reshape(hk, (b - a) * g, dq)
        po, pt, pl, _ = [x if x is None else x.view(hk, b - a, g, -1).transpose(0, 1) for x in _part(rows, k, v)]
        m = torch.maximum(top[a:b], pt)
        x, y = (top[a:b] - m).exp(), (pt - m).exp()
        o[a:b], total[a:b], top[a:b] = o[a:b] * x + po * y, total[a:b] * x + pl * y, m
    s["out"].copy_((o / total).view(n, hq, dv))
    if not case["weigh"]:
        return s["out"]
    w = (scores.sub_(top).exp_() / total).sum(dim=2)  # of the query heads of a KV head
    if case["weigh"] == "one":
        w = w.sum(dim=1, keepdim=True)
    at = at[:, None].expand(-1, w.shape[1], -1)
    seen = seen[:, None].expand_as(at)
    # entries behind a request's length repeat its first one and add nothing to it
    new = torch.where(seen, w + (case["decay"] - 1.0) * s["weights"].gather(2, at), 0.0)
    s["weights"].scatter_add_(2, at, new)
    return [s["out"], s["weights"]]


def _plain_evict(s):
    case = s["case"]
    lens, w, keep = s["lens"], s["weights"], case["keep"]
    n, lists, cap = w.shape
    at = torch.arange(cap, device="cuda")
    inside = (at < lens[:, None])[:, None].expand_as(w)
    sure = ((at < case["first"]) | (at >= lens[:, None] - case["recent"]))[:, None]
    key = torch.where(inside, torch.where(sure, math.inf, w), -math.inf)
    # a stable sort: of equal weights the earlier entry stays
    chosen = torch.zeros_like(inside).scatter_(2, key.argsort(dim=2, descending=True, stable=True)[..., :keep], True) & inside
    kept = torch.where(chosen, at, cap).sort(dim=2).values[..., : min(keep, cap)]
    i = at[: kept.shape[2]]
    src = torch.where(kept < cap, kept, i)  # a request within its budget: everything stays
    moved = torch.where(kept < cap, w.gather(2, src), 0.0)
    s["weights_out"].copy_(torch.where(inside, 0.0, s["weights_out"]))
    s["weights_out"][..., : kept.shape[2]] = torch.where(kept < cap, moved, s["weights_out"][..., : kept.shape[2]])
    torch.minimum(lens, torch.full_like(lens, keep), out=s["lens_out"])
    flat = s["pages"].view(-1, lists, _record(case) // lists)
    page = case["page"]
    rows = s["table"].long()[:, None].expand(-1, lists, -1).gather(2, src // page) * page + src % page
    to = (s["table"].long().gather(1, (i // page).expand(n, -1)) * page + i % page)[:, None].expand_as(rows)
    heads = torch.arange(lists, device="cuda")[None, :, None].expand_as(rows)
    flat[to, heads] = flat[rows, heads]
    return [s["pages"], s["weights_out"], s["lens_out"]]


def run(s):
    if own:
        case, kv = s["case"], s["kv"]
        if case["op"] == "norm":
            kv.append(s["k"], s.get("v"), s["cu"], s["start"], rope=s["rope"], rope_pos=s["at"], q=s["q"], q_out=s["q_out"],
                      q_weight=s.get("q_weight"), k_weight=s["k_weight"], eps=EPS)
            return [s["pages"], s["q_out"]]
        if case["op"] == "prefix":
            out = kv.prefix_attn(s["q"], s["lens"], groups=s["groups"], prefix=s["prefix"], weights=s.get("weights"),
                                 decay=case["decay"], out=s["out"])
            return [out, s["weights"]] if case["weigh"] else out
        kv.evict(s["lens"], s["weights"], case["keep"], first=case["first"], recent=case["recent"],
                 weights_out=s["weights_out"], lens_out=s["lens_out"])
        return [s["pages"], s["weights_out"], s["lens_out"]]
    return {"norm": _plain_norm, "prefix": _plain_prefix, "evict": _plain_evict}[s["case"]["op"]](s)


# ---- from the definitions, in 64 bits ----------------------------------------------------------


def _exact_norm(s, case, place):
    latent, half, first = case["layout"] == "latent", case["rotary"] // 2, case["first"] % 512
    place_of = [place(r, first + i) for r, c in enumerate(_counts(case)) for i in range(c)]
    at = s["at"].cpu().double().view(case["tokens"], -1)
    phase = torch.stack([torch.polar(torch.ones(()).double(), at[:, a] * f) for a, f in zip(s["axis"], s["freq"])], dim=1)
    phase = phase.cuda()[:, None]

    def turn(x, lo):
        x = x.clone()
        part = x[..., lo : lo + 2 * half]
        pairs = part.unflatten(-1, (half, 2)) if case["interleaved"] else part.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * phase)
        x[..., lo : lo + 2 * half] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        return x

    def norm(x, weight):
        x = x.double()
        return weight.double() * x / torch.sqrt((x * x).sum(dim=-1, keepdim=True) / x.shape[-1] + EPS)

    if latent:
        dv = case["dim_v"]
        rec = turn(torch.cat([norm(s["k"][..., :dv], s["k_weight"]), s["k"][..., dv:].double()], dim=-1), dv)
        q = s["q"].double()
    else:
        rec = torch.cat([turn(norm(s["k"], s["k_weight"]), 0), s["v"].double()], dim=-1)
        q = norm(s["q"], s["q_weight"])
    cache = s["pages"].double()
    cache.view(-1, _record(case))[torch.tensor(place_of, device="cuda")] = rec.flatten(1)
    return [cache, turn(q, 0)]


def _exact_prefix(s, case, place):
    hq, hk, dq, dv = (case[x] for x in ("q_heads", "kv_heads", "dim_qk", "dim_v"))
    lead, pre = _shared(case)
    owned = _ragged(case["requests"], case["own"])
    flat = s["pages"].view(-1, _record(case))
    out = torch.zeros((case["requests"], hq, dv), dtype=torch.float64, device="cuda")
    sums = s["weights"].double() if case["weigh"] else None
    for r, (p, o) in enumerate(zip(pre, owned)):
        rows = flat[torch.tensor([place(lead[r], x) for x in range(p)] + [place(r, p + x) for x in range(o)], device="cuda")]
        if case["weigh"]:
            sums[r, :, p : p + o] *= case["decay"]
        for h in range(hk):
            w = dq + dv
            kv = rows if case["layout"] == "latent" else rows[:, h * w : (h + 1) * w]
            k = kv[:, :dq].double()
            v = k[:, :dv] if case["layout"] == "latent" else kv[:, dq:].double()
            heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
            weight = torch.softmax(s["q"][r, heads].double() @ k.T / math.sqrt(dq), dim=1)
            out[r, heads] = weight @ v
            if case["weigh"]:
                sums[r, h if case["weigh"] == "heads" else 0, p : p + o] += weight[:, p:].sum(dim=0)
    return [out, sums] if case["weigh"] else out


def _exact_evict(s, case, place):
    pages, new = s["pages"].double(), s["weights_out"].double()
    lists = _lists(case, "lists")
    width = _record(case) // lists
    for r, length in enumerate(_contexts(case)):
        for x in range(lists):
            w = s["weights"][r, x].tolist()
            kept = set(range(min(case["first"], length))) | set(range(max(0, length - case["recent"]), length))
            rest = sorted((p for p in range(length) if p not in kept), key=lambda p: (-w[p], p))
            kept = sorted(kept | set(rest[: max(0, case["keep"] - len(kept))])) if length > case["keep"] else range(length)
            new[r, x, :length] = 0.0
            new[r, x, : len(kept)] = torch.tensor([w[p] for p in kept], dtype=torch.float64)
            go = [(place(r, i), place(r, p)) for i, p in enumerate(kept) if i != p]
            if go:
                to, at = torch.tensor(go, device="cuda").T
                cols = slice(x * width, (x + 1) * width)
                pages.view(-1, _record(case))[to, cols] = s["pages"].view(-1, _record(case))[at, cols].double()
    return [pages, new, None]


def exact(case, seed):
    s = prepare(case, seed)
    table, page = s["table"].cpu().tolist(), case["page"]
    place = lambda r, p: table[r][p // page] * page + p % page  # noqa: E731
    return {"norm": _exact_norm, "prefix": _exact_prefix, "evict": _exact_evict}[case["op"]](s, case, place)
