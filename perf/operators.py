"""Measured cases of the speculative-decoding operators: rotate-and-append to a paged cache, attention for a
tree of drafted tokens over it, and keeping the accepted path.

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


def listed():
    return [
        # one user, a short chat and a chain of four drafts: latency alone counts
        dict(GQA, name="tree_one_short", op="tree", requests=1, nodes=4, context=1000, ragged=False, page=64, select=0),
        # the batch-16 decode step of the benchmark (2048 selected rows of a 4096-row buffer), 8 drafts a request
        dict(GQA, name="tree_select_b16", op="tree", requests=16, nodes=8, context=4096, ragged=False, page=64,
             select=2048),
        # long documents without a selection: the cache's bytes are everything
        dict(GQA, name="tree_long_b4", op="tree", requests=4, nodes=16, context=131072, ragged=False, page=64, select=0),
        # a ragged batch with wide trees: as much arithmetic as memory
        dict(GQA, name="tree_wide_b8", op="tree", requests=8, nodes=64, context=16384, ragged=True, page=16, select=0),
        # the shared-latent batch of the benchmark with 8 drafts a request
        dict(LATENT, name="tree_latent_select_b8", op="tree", requests=8, nodes=8, context=4096, ragged=False, page=64,
             select=2048),
        # shared latent, dense and ragged, few drafts
        dict(LATENT, name="tree_latent_b4", op="tree", requests=4, nodes=5, context=32768, ragged=True, page=64, select=0),
        # one token a request appended with its query rotated: a decode step of batch 16
        dict(GQA, name="append_step_b16", op="append", requests=16, tokens=16, first=131000, page=64, with_q=True,
             drafts=False, rotary=128, interleaved=False),
        # a prefill chunk of four ragged prompts far into long contexts
        dict(GQA, name="append_chunk", op="append", requests=4, tokens=16384, first=1000000, page=64, with_q=True,
             drafts=False, rotary=128, interleaved=False),
        # shared-latent prefill chunk: the latents and the queries' rotary part
        dict(LATENT, name="append_latent_chunk", op="append", requests=5, tokens=8191, first=777, page=64, with_q=True,
             drafts=False, rotary=64, interleaved=True),
        # trees of 64 drafts for 32 requests: every node's angle goes by its depth
        dict(GQA, name="append_drafts_b32", op="append", requests=32, tokens=2048, first=50000, page=16, with_q=True,
             drafts=True, rotary=64, interleaved=False),
        # accepted paths of up to 6 of 8 drafts
        dict(GQA, name="keep_b16", op="keep", requests=16, nodes=8, accepted=6, first=4000, page=64),
        # accepted paths of up to 16 of 64 drafts in a large batch
        dict(GQA, name="keep_b256", op="keep", requests=256, nodes=64, accepted=16, first=500, page=16),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "append", "append", "keep"])
    shape = dict(rng.choice([GQA, GQA, LATENT]))
    latent = shape["layout"] == "latent"
    if not latent:
        shape["kv_heads"] = rng.choice([2, 4, 8])
        shape["q_heads"] = shape["kv_heads"] * rng.choice([1, 2, 4, 5, 7, 8])
        shape["dim_qk"] = shape["dim_v"] = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "tree":
        nodes = _spread(rng, 1, 12 if latent else 64)
        context = _spread(rng, 1, 65536)
        select = min(context, rng.choice([0, 0, 512, 2048]))
        entries = select or context
        most = max(1, min(32, (1 << 31) // max(1, entries * nodes * shape["q_heads"] * (shape["dim_qk"] + shape["dim_v"])),
                          (1 << 19) // entries))
        return dict(shape, op=op, requests=_spread(rng, 1, most) if most > 1 else 1, nodes=nodes, context=context,
                    ragged=rng.random() < 0.5, page=page, select=select)
    if op == "append":
        drafts = rng.random() < 0.3
        requests = _spread(rng, 1, 64)
        tokens = requests * _spread(rng, 1, 64) if drafts else _spread(rng, 1, 8192)
        rotary = 64 if latent else rng.choice([32, 64, shape["dim_qk"]])
        return dict(shape, op=op, requests=requests, tokens=tokens, first=_spread(rng, 1, 1 << 20), page=page,
                    with_q=rng.random() < 0.7, drafts=drafts, rotary=rotary, interleaved=rng.random() < 0.5)
    nodes = _spread(rng, 1, 64)
    return dict(shape, op=op, requests=_spread(rng, 1, 256), nodes=nodes, accepted=_spread(rng, 1, nodes),
                first=_spread(rng, 1, 2000), page=page)


# ---- sizes that go by the case alone -----------------------------------------------------------


def _record(case):
    if case["layout"] == "latent":
        return case["dim_qk"]
    return case["kv_heads"] * (case["dim_qk"] + case["dim_v"])


def _lens(case):
    """Context length of each request: all the same, or spread from an eighth of the largest to it."""
    n, top = case["requests"], case["context"]
    if not case["ragged"] or n == 1:
        return [top] * n
    return [max(1, top // 8 + (top - top // 8) * r // (n - 1) - (r * 5) % 7 * (r < n - 1)) for r in range(n)]


def _counts(case):
    """Tokens each request appends: equal trees, or a ragged split (some may append nothing)."""
    n, total = case["requests"], case["tokens"]
    if case["drafts"]:
        return [total // n] * n
    cuts = [total * (r + (r % 3) * (0 < r)) // (n + 2) for r in range(n)] + [total]
    cuts = sorted(min(c, total) for c in cuts) if total > n else [min(r, total) for r in range(n + 1)]
    cuts[0], cuts[-1] = 0, total
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _kept(case):
    """Accepted nodes of each request: from none to `accepted`."""
    return [r % (case["accepted"] + 1) if case["requests"] > 1 else case["accepted"] for r in range(case["requests"])]


def _trees(case, count):
    """Parents of a request's nodes, -1 for a child of the last context token: chains and bushes by turns."""
    rng = random.Random(7 * count + case["requests"])
    return [[-1] + [j - 1 if r % 3 == 0 else rng.randrange(-1, j) for j in range(1, count)] for r in range(case["requests"])]


def work(case):
    rec = 2 * _record(case)
    if case["op"] == "tree":
        lens = _lens(case)
        rows = [min(case["select"], n) if case["select"] else n for n in lens]
        t, hq = case["nodes"], case["q_heads"]
        bytes_ = sum(rows) * rec + case["requests"] * (t * rec + 2 * t * hq * (case["dim_qk"] + case["dim_v"]) + 16 * t)
        if case["select"]:
            bytes_ += 4 * sum(rows)
        flops = sum(2 * t * hq * (case["dim_qk"] + case["dim_v"]) * (n + 1) for n in rows)
        return {"bytes": bytes_, "flops": flops}
    if case["op"] == "append":
        width = case["rotary"] if case["layout"] == "latent" else case["dim_qk"]
        q = case["q_heads"] * width if case["with_q"] else 0
        pairs = case["rotary"] // 2 * (case["kv_heads"] + (case["q_heads"] if case["with_q"] else 0))
        return {"bytes": case["tokens"] * (2 * rec + 4 * q + 8 * case["drafts"]), "flops": 6 * pairs * case["tokens"]}
    moved = sum(_kept(case))
    return {"bytes": 2 * moved * rec + 4 * moved, "flops": 0}


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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    n, hq, dq = case["requests"], case["q_heads"], case["dim_qk"]
    s = {"case": case}
    if case["op"] == "tree":
        t, lens = case["nodes"], _lens(case)
        s["pages"], s["table"] = _cache(case, max(lens) + t, g)
        s["lens"] = torch.tensor(lens, dtype=torch.int64, device="cuda")
        # heads from flat to peaked softmaxes
        sharp = torch.linspace(0.5, 3.0, hq, device="cuda").view(1, 1, hq, 1)
        s["q"] = (torch.randn((n, t, hq, dq), generator=g, device="cuda") * sharp).to(torch.bfloat16)
        masks = []
        for parents in _trees(case, t):
            seen = []
            for j, p in enumerate(parents):
                seen.append((seen[p] if p >= 0 else 0) | 1 << j)
            masks.append([[m - (1 << 64) if m >> 63 else m] for m in seen])
        s["mask"] = torch.tensor(masks, dtype=torch.int64, device="cuda")
        if case["select"]:
            # a shuffled list of distinct rows a request, -1 behind a short one
            key = torch.rand((n, case["context"]), generator=g, device="cuda")
            key.masked_fill_(torch.arange(case["context"], device="cuda") >= s["lens"][:, None], 2.0)
            score, rows = key.topk(case["select"], dim=1, largest=False)
            s["locs"] = torch.where(score < 2.0, rows, -1).to(torch.int32)
        s["out"] = torch.zeros((n, t, hq, case["dim_v"]), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "append":
        counts, total = _counts(case), case["tokens"]
        s["pages"], s["table"] = _cache(case, max(counts) + case["first"] % 512, g)
        s["cu"] = torch.tensor([sum(counts[:r]) for r in range(n + 1)], dtype=torch.int32, device="cuda")
        # the cache holds the last `first` % 512 positions and what comes; angles count from `first`
        s["start"] = torch.full((n,), case["first"] % 512, dtype=torch.int64, device="cuda")
        if case["drafts"]:
            depths = []
            for parents in _trees(case, total // n):
                d = []
                for p in parents:
                    d.append(d[p] + 1 if p >= 0 else 0)
                depths += d
            at = torch.tensor(depths, dtype=torch.int64, device="cuda")
        else:
            at = torch.cat([torch.arange(c, device="cuda") for c in counts])
        s["at"] = at + case["first"]
        # keys, values and queries as views of one projection, as a model has them
        kw = case["kv_heads"] * dq
        vw = 0 if case["layout"] == "latent" else case["kv_heads"] * case["dim_v"]
        width = case["rotary"] if case["layout"] == "latent" else dq
        qw = hq * width if case["with_q"] else 0
        flat = torch.randn((total, qw + kw + vw), generator=g, device="cuda", dtype=torch.bfloat16)
        if case["with_q"]:
            s["q"] = flat[:, :qw].unflatten(1, (hq, width))
            s["q_out"] = torch.empty((total, hq, width), dtype=torch.bfloat16, device="cuda")
        s["k"] = flat[:, qw : qw + kw].unflatten(1, (case["kv_heads"], dq))
        if vw:
            s["v"] = flat[:, qw + kw :].unflatten(1, (case["kv_heads"], case["dim_v"]))
        half = case["rotary"] // 2
        s["freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        s["freq_gpu"] = s["freq"].cuda()
    else:
        t, kept = case["nodes"], _kept(case)
        s["pages"], s["table"] = _cache(case, case["first"] + t, g)
        s["lens"] = torch.full((n,), case["first"], dtype=torch.int64, device="cuda") - torch.arange(n, device="cuda") % min(
            case["first"], 7)
        # ascending nodes: an accepted path never goes back
        order = torch.rand((n, t), generator=g, device="cuda").argsort(dim=1)[:, : case["accepted"]]
        count = torch.tensor(kept, dtype=torch.int32, device="cuda")
        col = torch.arange(case["accepted"], device="cuda")
        path = torch.where(col < count[:, None], order, t).sort(dim=1).values
        s["path"] = torch.where(path < t, path, 0).to(torch.int32)
        s["count"] = count
    if own:
        from hierarchical_kv_cache_02_gb300 import PagedKV, RopeTable

        s["kv"] = PagedKV(_config(case), s["pages"], s["table"])
        if case["op"] == "append":
            s["rope"] = RopeTable(case["rotary"], inv_freq=s["freq"].tolist(), interleaved=case["interleaved"])
    return s


# ---- plain forms -------------------------------------------------------------------------------


def _rows_of(s, positions):
    """Flat row of each position [requests][n] in the cache seen as [rows][record]."""
    page = s["case"]["page"]
    return s["table"].long().gather(1, positions // page) * page + positions % page


def _bits(mask, t):
    return (mask.repeat_interleave(64, dim=2)[:, :, :t] >> (torch.arange(t, device="cuda") % 64)) & 1 == 1


def _plain_tree(s):
    case = s["case"]
    n, t, hq, hk, dq, dv = (case[x] for x in ("requests", "nodes", "q_heads", "kv_heads", "dim_qk", "dim_v"))
    lens = s["lens"]
    if case["select"]:
        seen = s["locs"] >= 0
        at = s["locs"].long().clamp(min=0)
    else:
        at = torch.arange(case["context"], device="cuda").expand(n, -1)
        seen = at < lens[:, None]
        at = torch.minimum(at, lens[:, None])
    at = torch.cat([at, lens[:, None] + torch.arange(t, device="cuda")], dim=1)
    rows = s["pages"].view(-1, _record(case))[_rows_of(s, at)]
    e = at.shape[1]
    if case["layout"] == "latent":
        k = rows.float().view(n, e, 1, dq).transpose(1, 2)
        v = k[..., :dv]
    else:
        rows = rows.view(n, e, hk, dq + dv).transpose(1, 2)
        k, v = rows[..., :dq].float(), rows[..., dq:].float()
    g = hq // hk
    q = s["q"].float().view(n, t, hk, g, dq).permute(0, 2, 1, 3, 4).reshape(n, hk, t * g, dq)
    a = q @ k.transpose(2, 3)
    a *= 1.0 / math.sqrt(dq)
    ok = torch.cat([seen[:, None, :].expand(n, t, -1), _bits(s["mask"], t)], dim=2)
    a.view(n, hk, t, g, e).masked_fill_(~ok[:, None, :, None, :], -math.inf)
    top = a.amax(dim=3, keepdim=True).clamp(min=-3e38)
    a.sub_(top).exp_()
    total = a.sum(dim=3, keepdim=True)
    o = (a @ v) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(o.view(n, hk, t, g, dv).permute(0, 2, 1, 3, 4).reshape(n, t, hq, dv))
    return s["out"]


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


def _plain_append(s):
    case = s["case"]
    total = case["tokens"]
    t = torch.arange(total, device="cuda")
    req = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    at = s["start"][req] + t - s["cu"][req]
    angle = s["at"].double()[:, None] * s["freq_gpu"]  # 64 bits: far positions turn many times
    cos, sin = angle.cos().float(), angle.sin().float()
    latent = case["layout"] == "latent"
    rec = _turned(s["k"].float(), cos, sin, case["dim_v"] if latent else 0, case["interleaved"]).to(torch.bfloat16)
    if not latent:
        rec = torch.cat([rec, s["v"]], dim=2)
    page = case["page"]
    row = s["table"][req, at // page].long() * page + at % page
    s["pages"].view(-1, _record(case))[row] = rec.reshape(total, -1)
    if case["with_q"]:
        s["q_out"].copy_(_turned(s["q"].float(), cos, sin, 0, case["interleaved"]))
        return [s["pages"], s["q_out"]]
    return [s["pages"]]


def _plain_keep(s):
    flat = s["pages"].view(-1, _record(s["case"]))
    i = torch.arange(s["path"].shape[1], device="cuda")
    src = _rows_of(s, s["lens"][:, None] + s["path"].long())
    dst = _rows_of(s, s["lens"][:, None] + i)
    dst = torch.where(i < s["count"][:, None], dst, dst[:, :1])
    src = torch.where(i < s["count"][:, None], src, src[:, :1])
    # entries behind a path repeat its first move; a request without a path keeps its row
    src = torch.where(s["count"][:, None] > 0, src, dst)
    flat[dst.reshape(-1)] = flat[src.reshape(-1)]
    return s["pages"]


def run(s):
    if own:
        case = s["case"]
        if case["op"] == "tree":
            return s["kv"].tree_attn(s["q"], s["lens"], s["mask"], locs=s.get("locs"), out=s["out"])
        if case["op"] == "append":
            s["kv"].append(s["k"], s.get("v"), s["cu"], s["start"], rope=s["rope"], rope_pos=s["at"], q=s.get("q"),
                           q_out=s.get("q_out"))
            return [s["pages"], s["q_out"]] if case["with_q"] else [s["pages"]]
        s["kv"].keep_path(s["lens"], s["path"], s["count"])
        return s["pages"]
    return {"tree": _plain_tree, "append": _plain_append, "keep": _plain_keep}[s["case"]["op"]](s)


# ---- from the definitions, in 64 bits ----------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    pages, table, page = s["pages"], s["table"].cpu().tolist(), case["page"]
    n = case["requests"]
    place = lambda r, p: table[r][p // page] * page + p % page  # noqa: E731
    flat = pages.view(-1, _record(case))
    if case["op"] == "tree":
        hq, hk, dq, dv, t = (case[x] for x in ("q_heads", "kv_heads", "dim_qk", "dim_v", "nodes"))
        out = torch.zeros((n, t, hq, dv), dtype=torch.float64, device="cuda")
        masks = s["mask"][:, :, 0].tolist()
        for r, length in enumerate(_lens(case)):
            at = [p for p in s["locs"][r].tolist() if p >= 0] if case["select"] else range(length)
            idx = torch.tensor([place(r, p) for p in list(at) + list(range(length, length + t))], device="cuda")
            rows = flat[idx]
            hidden = torch.tensor([[masks[r][i] >> j & 1 == 0 for j in range(t)] for i in range(t)], device="cuda")
            for h in range(hq):
                w = dq + dv
                kv = rows if case["layout"] == "latent" else rows[:, h // (hq // hk) * w :][:, :w]
                k = kv[:, :dq].double()
                v = k[:, :dv] if case["layout"] == "latent" else kv[:, dq:].double()
                a = s["q"][r, :, h].double() @ k.T / math.sqrt(dq)
                a[:, len(at) :][hidden] = -math.inf
                out[r, :, h] = torch.softmax(a, dim=1) @ v
        return out
    if case["op"] == "append":
        latent = case["layout"] == "latent"
        half = case["rotary"] // 2
        place_of = []
        first = case["first"] % 512
        for r, c in enumerate(_counts(case)):
            place_of += [place(r, first + i) for i in range(c)]
        phase = torch.polar(torch.ones(()).double(), torch.outer(s["at"].cpu().double(), s["freq"])).cuda()[:, None]

        def turn(x, lo):
            x = x.double().clone()
            part = x[..., lo : lo + 2 * half]
            pairs = part.unflatten(-1, (half, 2)) if case["interleaved"] else part.unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * phase)
            x[..., lo : lo + 2 * half] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
            return x

        rec = turn(s["k"], case["dim_v"] if latent else 0)
        if not latent:
            rec = torch.cat([rec, s["v"].double()], dim=-1)
        cache = pages.double()
        cache.view(-1, _record(case))[torch.tensor(place_of, device="cuda")] = rec.flatten(1)
        return [cache, turn(s["q"], 0)] if case["with_q"] else [cache]
    moved = pages.clone().view(-1, _record(case))
    path, lens = s["path"].tolist(), s["lens"].tolist()
    to = [(place(r, lens[r] + i), place(r, lens[r] + path[r][i])) for r, c in enumerate(_kept(case)) for i in range(c)]
    if to:
        a, b = torch.tensor(to, device="cuda").T
        moved[a] = flat[b]
    return moved.view_as(pages).double()
