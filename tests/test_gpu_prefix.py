"""Attention over shared prefixes on the GPU, and the weights it sums up, against a plain 64-bit form; and a decode step of
all operators of a batch together."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import batch_ref as ref
from hierarchical_kv_cache_02_gb300 import DEVERR_LOC, DEVERR_PAGE, HsError, PagedKV, RopeTable
from spec_ref import U_FP32, row_of
from test_gpu_batch import DEV, gen, gqa, make_cache, mla


def shared_of(R, groups, prefix):
    """For each request the first of its group and what it shares."""
    lead, pre = list(range(R)), [0] * R
    for g, p in enumerate(prefix):
        for r in range(groups[g], groups[g + 1]):
            lead[r], pre[r] = groups[g], p
    return lead, pre


def rows_of(kv, lead, pre, lens):
    t = kv.table.cpu() if kv.table is not None else None
    flat = kv.pages.view(-1, kv.cfg.record_elems)
    page, most = kv.pages.shape[1], kv._kv.max_pages
    out = []
    for r, n in enumerate(lens):
        idx = [row_of(t, lead[r] if p < pre[r] else r, p, page, most) for p in range(n)] if n >= pre[r] else []
        out.append(flat[torch.tensor(idx, dtype=torch.int64, device=DEV)])
    return out


def check(cfg, groups, prefix, lens, page=16, lists=0, decay=1.0, table=True, seed=0, scale=None, only=None, kv=None, q=None, errors=0,
          slack=0, stream=None):
    """Every request has pages of its own for all its positions: shared ones have to come from the first of its group."""
    R, Hq = cfg.num_requests, cfg.num_q_heads
    kv = kv or make_cache(cfg, max(max(lens), 1) + slack, page, seed, table)
    if q is None:
        q = torch.randn((R, Hq, cfg.head_dim_qk), generator=gen(seed + 5), device=DEV)
        q = (q * torch.linspace(0.3, 3.0, Hq, device=DEV)[:, None]).to(torch.bfloat16)
    lead, pre = shared_of(R, groups, prefix)
    lt = torch.tensor(lens, dtype=torch.int64, device=DEV)
    gt = torch.tensor(groups, dtype=torch.int32, device=DEV)
    pt = torch.tensor(prefix, dtype=torch.int64, device=DEV)
    cap = max(max(lens), 1) + slack
    acc = torch.rand((R, lists, cap), generator=gen(seed + 6), device=DEV) if lists else None
    before = acc.clone() if lists else None
    out = torch.full((R, Hq, cfg.head_dim_v), 7.0, dtype=torch.bfloat16, device=DEV)
    got = kv.prefix_attn(q, lt, groups=gt, prefix=pt, weights=acc, decay=decay, out=out, scale=scale, stream=stream)
    assert got is out and kv.errors(reset=True) == errors
    own = [max(0, n - p) for n, p in zip(lens, pre)]
    want, bound, weights = ref.attention(cfg, rows_of(kv, lead, pre, lens), q, cfg.default_scale if scale is None else scale, own, only)
    err = (out.double() - want).abs()
    assert bool(torch.isfinite(out.double()).all()), "not finite"
    assert bool((err <= bound).all()), (float((err - bound).max()), (err > bound).nonzero()[:4].tolist())
    if lists:
        for r in range(R):
            a, b = (pre[r], lens[r]) if lens[r] >= pre[r] else (0, 0)
            w = weights[r][:, :, : b - a].unflatten(1, (lists, Hq // lists)).sum(dim=2)
            new = decay * before[r, :, a:b].double() + w[0]
            off = w[1] + (Hq // lists + 3) * U_FP32 * (new.abs() + abs(decay) * before[r, :, a:b].double())
            e = (acc[r, :, a:b].double() - new).abs()
            assert bool((e <= off).all()), (r, float((e - off).max()))
            assert ref.same(acc[r, :, :a], before[r, :, :a]) and ref.same(acc[r, :, b:], before[r, :, b:])
    return kv, q, out, acc


SHAPES = [
    pytest.param(lambda R: gqa(R), id="gqa"),
    pytest.param(lambda R: gqa(R, 28, 4, 64), id="gqa64-group-of-7"),
    pytest.param(lambda R: gqa(R, 4, 4), id="gqa-ungrouped"),
    pytest.param(lambda R: gqa(R, 40, 2), id="gqa-group-of-20"),
    pytest.param(lambda R: gqa(R, 128, 1), id="gqa-group-of-128"),
    pytest.param(lambda R: mla(R), id="mla"),
    pytest.param(lambda R: mla(R, 16), id="mla-16-heads"),
    pytest.param(lambda R: mla(R, 130), id="mla-130-heads"),
    pytest.param(lambda R: gqa(R, 4, 2, 80), id="any-80"),
    pytest.param(lambda R: gqa(R, 4, 2, 192, 128), id="any-192-128"),
    pytest.param(lambda R: gqa(R, 2, 1, 576), id="any-576"),
    pytest.param(lambda R: gqa(R, 130, 1, 64), id="any-group-of-130"),
    pytest.param(lambda R: mla(R, 4, 128, 64), id="any-latent-128-64"),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("R,groups,prefix,lens,page", [
    (1, [0], [], [1], 16),
    (1, [0], [], [300], 64),
    (4, [0], [], [0, 1, 129, 128], 16),
    (2, [0, 2], [100], [130, 101], 16),
    (3, [0, 3], [32], [32, 33, 400], 32),
    (5, [1, 4], [257], [40, 258, 400, 257, 0], 7),
    (6, [0, 2, 2, 3, 6], [64, 5, 50, 31], [64, 100, 60, 40, 500, 31], 16),
    (7, [0, 7], [1], [1, 2, 3, 4, 5, 6, 0], 1),
    (2, [0, 2], [0], [70, 7], 16),
])
@pytest.mark.parametrize("lists", [0, 1, 2])
def test_prefixes(shape, R, groups, prefix, lens, page, lists):
    cfg = shape(R)
    if lists == 2:
        if cfg.num_kv_heads == 1:
            pytest.skip("one list either way")
        lists = cfg.num_kv_heads
    check(cfg, groups, prefix, lens, page, lists=lists, decay=0.75 if lists else 1.0, seed=R + sum(lens))


@pytest.mark.parametrize("cfg,groups,prefix,most,page", [
    (gqa(40), [0, 40], 3000, 300, 64), (gqa(70), [0, 66], 5000, 200, 16), (gqa(33, 8, 2, 64), [2, 9, 30], 900, 1100, 32),
    (gqa(300, 4, 2), [0, 130, 290], 700, 90, 16), (gqa(700, 2, 1), [0], 0, 150, 16), (gqa(600, 2, 1, 64), [0, 600], 40, 60, 32),
    (gqa(3), [0, 2], 20000, 9000, 16), (gqa(5, 32, 8, 64), [0, 5], 9000, 3, 128), (gqa(130, 20, 4), [0, 60, 128], 333, 140, 48),
    (gqa(1500, 2, 1), list(range(0, 1401, 2)), 90, 40, 16), (gqa(1100, 2, 1, 80), list(range(3, 1100, 3)), 50, 30, 16), (mla(1100, 4), list(range(1, 1001, 4)), 70, 40, 32),
    (mla(20), [0, 17], 3000, 300, 64), (mla(5), [0, 2], 9000, 4000, 16), (mla(90, 16), [0, 40, 90], 700, 100, 16), (mla(300, 4), [0, 200], 90, 40, 32),
])
@pytest.mark.parametrize("weigh", [False, True])
def test_many_tiles_and_requests_a_worker(cfg, groups, prefix, most, page, weigh):
    """Workers that walk through many tiles, items and requests, empty ones among them; a sample of the rows is compared."""
    R, Hq = cfg.num_requests, cfg.num_q_heads
    g = torch.Generator().manual_seed(R)
    prefix = [max(0, prefix - 11 * x) for x in range(len(groups) - 1)]
    lead, pre = shared_of(R, groups, prefix)
    lens = [p + int(torch.randint(0, most, (1,), generator=g)) if r % 9 != 5 else 0 for r, p in enumerate(pre)]
    lens[0] = pre[0] + most
    pick = torch.randint(0, 10**9, (200, 2), generator=g).tolist()
    only = {(a % R, b % Hq) for a, b in pick} | {(0, Hq - 1), (R - 1, 0)}
    check(cfg, groups, prefix, lens, page, lists=cfg.num_kv_heads if weigh else 0, only=only, seed=R)


def test_without_a_table_and_without_groups():
    for cfg in (gqa(3), mla(3), gqa(3, 4, 2, 80)):
        check(cfg, [0, 2], [50], [60, 70, 200], 16, table=False, lists=1)
        kv, q, out, _ = check(cfg, [0], [], [60, 70, 200])
        lens = torch.tensor([60, 70, 200], dtype=torch.int64, device=DEV)
        assert ref.same(kv.prefix_attn(q, lens), out)


@pytest.mark.parametrize("cfg", [gqa(4), gqa(4, 8, 2, 64), mla(4), gqa(4, 4, 2, 80)], ids=["gqa", "gqa64", "mla", "any"])
@pytest.mark.parametrize("scale", [0.0, -0.07, 0.5])
def test_scales(cfg, scale):
    check(cfg, [0, 3], [200], [300, 201, 200, 150], scale=scale, lists=1)


@pytest.mark.parametrize("cfg", [gqa(4), gqa(4, 8, 2, 64), mla(4), gqa(4, 4, 2, 80)], ids=["gqa", "gqa64", "mla", "any"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_a_request_does_not_see_has_no_influence(cfg, bad):
    """Everything that nobody reads, and what one request alone sees, of NaN or infinities: the others' results are those of a clean
    cache, bit for bit."""
    groups, prefix, lens = [0, 3], [150], [170, 230, 300, 77]
    kv, q, clean, acc = check(cfg, groups, prefix, lens, lists=1, slack=40)
    lead, pre = shared_of(4, groups, prefix)
    flat, t = kv.pages.view(-1, cfg.record_elems), kv.table.cpu()
    good = [row_of(t, lead[r] if p < pre[r] else r, p, 16, 0) for r in (0, 1, 3) for p in range(lens[r])]
    sick = torch.ones(flat.shape[0], dtype=torch.bool, device=DEV)
    sick[torch.tensor(good, device=DEV)] = False
    flat[sick] = bad
    again = torch.rand(acc.shape, generator=gen(6), device=DEV)
    out = kv.prefix_attn(q, torch.tensor(lens, device=DEV), groups=torch.tensor(groups, dtype=torch.int32, device=DEV),
                         prefix=torch.tensor(prefix, device=DEV), weights=again)
    for r in (0, 1, 3):
        assert ref.same(out[r], clean[r]) and ref.same(again[r], acc[r])
    assert bool((~torch.isfinite(out[2].double())).any(dim=-1).all())  # its own positions are sick: every head sees it


@pytest.mark.parametrize("cfg", [gqa(3), mla(3), gqa(3, 4, 2, 80)], ids=["gqa", "mla", "any"])
def test_a_value_that_is_infinite_reaches_who_sees_it(cfg):
    kv, q, clean, _ = check(cfg, [0, 2], [100], [120, 130, 140])
    t = kv.table.cpu()
    dv = cfg.head_dim_v
    at = 0 if cfg.layout == 0 else cfg.head_dim_qk
    kv.pages.view(-1, cfg.record_elems)[row_of(t, 1, 110, 16, 0), at + 3] = float("nan")  # request 1's own
    out = kv.prefix_attn(q, torch.tensor([120, 130, 140], device=DEV), groups=torch.tensor([0, 2], dtype=torch.int32, device=DEV),
                         prefix=torch.tensor([100], device=DEV))
    assert ref.same(out[0], clean[0]) and ref.same(out[2], clean[2])
    G = cfg.num_q_heads // cfg.num_kv_heads
    assert bool(torch.isnan(out[1, :G, 3]).all())
    if cfg.layout == 1:  # a value alone, no key: the other dims and heads are as they were
        keep = torch.ones((cfg.num_q_heads, dv), dtype=torch.bool, device=DEV)
        keep[:G, 3] = False
        assert ref.same(out[1][keep], clean[1][keep])


@pytest.mark.parametrize("cfg", [gqa(4), gqa(4, 8, 2, 64), mla(4), gqa(4, 4, 2, 80)], ids=["gqa", "gqa64", "mla", "any"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_score_that_is_no_number_reaches_who_sees_it(cfg, bad):
    """In a key that a group shares, in one of a request's own, and in the only one that a request sees."""
    groups, prefix, lens = [0, 2], [150], [170, 330, 260, 1]
    kv, q, clean, _ = check(cfg, groups, prefix, lens)
    flat, t = kv.pages.view(-1, cfg.record_elems), kv.table.cpu()
    G = cfg.num_q_heads // cfg.num_kv_heads
    for r, p, who in ((0, 20, (0, 1)), (1, 300, (1,)), (2, 70, (2,)), (3, 0, (3,))):
        row = row_of(t, r, p, 16, 0)
        keep = flat[row].clone()
        flat[row, :G] = bad  # of the first KV head
        out = kv.prefix_attn(q, torch.tensor(lens, device=DEV), groups=torch.tensor(groups, dtype=torch.int32, device=DEV),
                             prefix=torch.tensor(prefix, device=DEV))
        flat[row] = keep
        for x in range(4):
            if x not in who:
                assert ref.same(out[x], clean[x])
            elif bad != bad:
                assert bool(torch.isnan(out[x, :G]).all())
            assert ref.same(out[x, G:], clean[x, G:])
    assert kv.errors() == 0


@pytest.mark.parametrize("cfg", [gqa(3), gqa(3, 8, 2, 64), mla(3), gqa(3, 4, 2, 80)], ids=["gqa", "gqa64", "mla", "any"])
def test_scores_of_both_infinities(cfg):
    """Of one key: +infinity makes a row NaN, -infinity is a weight of zero; alone it gives zeros."""
    lens, sick, D = [70, 300, 1], 40, cfg.head_dim_qk
    q = torch.randn((3, cfg.num_q_heads, D), generator=gen(1), device=DEV).to(torch.bfloat16)
    q[..., D - 1] = torch.where(torch.arange(cfg.num_q_heads, device=DEV) % 2 == 0, 1.0, -1.0).to(torch.bfloat16)
    kv = make_cache(cfg, 300, 16, 5)
    flat, t = kv.pages.view(-1, cfg.record_elems), kv.table.cpu()
    width = cfg.record_elems // cfg.num_kv_heads
    for r, p in ((0, sick), (2, 0)):  # of every KV head; of a latent a value behind those of V
        flat[row_of(t, r, p, 16, 0), D - 1 :: width] = float("inf")
    out = kv.prefix_attn(q, torch.tensor(lens, device=DEV), groups=torch.tensor([0, 2], dtype=torch.int32, device=DEV),
                         prefix=torch.tensor([60], device=DEV))
    rows = [flat[torch.tensor([row_of(t, 0 if p < 60 and r < 2 else r, p, 16, 0) for p in range(n) if r == 2 or p != sick], device=DEV)]
            for r, n in enumerate(lens)]
    want, bound, _ = ref.attention(cfg, rows[:2] + [rows[2][:0]], q, cfg.default_scale, [0] * 3)
    assert bool(torch.isnan(out[:, ::2]).all())
    assert bool(((out.double() - want).abs() <= bound)[:, 1::2].all()) and torch.count_nonzero(out[2, 1::2]) == 0
    assert kv.errors() == 0


@pytest.mark.parametrize("cfg", [gqa(3), gqa(3, 8, 2, 64), mla(3), gqa(3, 4, 2, 80)], ids=["gqa", "gqa64", "mla", "any"])
def test_records_beyond_32_bits(cfg):
    """The same records in a small cache and in pages at both ends of one of 9 GB give the same bits throughout."""
    R, page, most = cfg.num_requests, 16, 208
    near = make_cache(cfg, most, page, 3)
    n = 9 * 10**9 // (2 * page * cfg.record_elems)
    pages = torch.empty((n, page, cfg.record_elems), dtype=torch.bfloat16, device=DEV)
    count = near.table.numel()
    ids = torch.cat([torch.arange(n - count + 4, n), torch.arange(4)])[torch.randperm(count, generator=torch.Generator().manual_seed(1))].to(DEV)
    pages[ids] = near.pages[near.table.flatten().long()]
    far = PagedKV(cfg, pages, ids.to(torch.int32).view_as(near.table))
    D, Dv, latent = cfg.head_dim_qk, cfg.head_dim_v, cfg.layout == 0
    k = torch.randn((R, cfg.num_kv_heads, D), generator=gen(1), device=DEV).to(torch.bfloat16)
    q = torch.randn((R, cfg.num_q_heads, D), generator=gen(2), device=DEV).to(torch.bfloat16)
    lens, cu = [180, 200, 77], torch.arange(R + 1, dtype=torch.int32, device=DEV)
    groups, prefix = torch.tensor([0, 2], dtype=torch.int32, device=DEV), torch.tensor([64], device=DEV)
    got = []
    for kv in (near, far):
        lt, acc = torch.tensor(lens, device=DEV), torch.zeros((R, 1, most), device=DEV)
        kv.append(k, None if latent else k[..., :Dv], cu, lt - 1, rope=RopeTable(16), k_weight=torch.ones(Dv if latent else D, device=DEV))
        out = kv.prefix_attn(q, lt, groups=groups, prefix=prefix, weights=acc)
        kv.evict(lt, acc, 100, first=64, recent=8, lens_out=lt)
        got.append((out, lt, acc, kv.pages[kv.table.flatten().long()]))
        assert kv.errors() == 0
    for a, b in zip(*got):
        assert ref.same(a, b)


@pytest.mark.parametrize("cfg", [gqa(5), mla(5), gqa(5, 4, 2, 80)], ids=["gqa", "mla", "any"])
def test_bad_lengths_groups_and_pages(cfg):
    def call(kv, q, lens, groups, prefix, acc=None):
        return kv.prefix_attn(q, torch.tensor(lens, dtype=torch.int64, device=DEV), groups=torch.tensor(groups, dtype=torch.int32, device=DEV),
                              prefix=torch.tensor(prefix, dtype=torch.int64, device=DEV), weights=acc)

    # a request shorter than its prefix, one of a negative length and one longer than its pages: zeros, the others as ever
    kv, q, good, acc = check(cfg, [0, 3], [50], [60, 70, 80, 0, 0], lists=1)
    w = torch.rand(acc.shape, generator=gen(6), device=DEV)
    w0 = w.clone()
    out = call(kv, q, [60, 49, 80, -1, 81], [0, 3], [50], w)
    assert kv.errors(reset=True) == DEVERR_LOC
    assert ref.same(out[[0, 2]], good[[0, 2]]) and torch.count_nonzero(out[[1, 3, 4]]) == 0
    assert ref.same(w[[0, 2]], acc[[0, 2]]) and ref.same(w[[1, 3, 4]], w0[[1, 3, 4]])
    # bounds that do not ascend or leave the requests: nothing is shared
    _, _, alone, _ = check(cfg, [0], [], [60, 70, 80, 0, 0], kv=kv, q=q)
    for groups in ([0, 3, 2], [-1, 3, 4], [0, 3, 6], [0, 5, 0, 5, 0, 5]):
        out = call(kv, q, [60, 70, 80, 0, 0], groups, [50] * (len(groups) - 1))
        assert kv.errors(reset=True) == DEVERR_LOC and ref.same(out, alone)
    # prefixes outside the pages share nothing either
    for p in (-1, 81, 1 << 40):
        out = call(kv, q, [60, 70, 80, 0, 0], [0, 3], [p])
        assert kv.errors(reset=True) == DEVERR_LOC and ref.same(out, alone)
    # weights with less room than a request has positions
    w = torch.zeros((5, 1, 65), device=DEV)
    full = torch.zeros((5, 1, 80), device=DEV)
    call(kv, q, [60, 70, 80, 0, 0], [0], [], w)
    assert kv.errors(reset=True) == DEVERR_LOC
    call(kv, q, [60, 70, 80, 0, 0], [0], [], full)
    assert kv.errors() == 0 and ref.same(w, full[:, :, :65])
    # table entries that are no pages: their positions are not seen
    kv.table[0, 1], kv.table[1, 4] = -1, 10**6
    w = torch.zeros((5, 1, 80), device=DEV)
    out = call(kv, q, [60, 70, 80, 0, 0], [0, 3], [50], w)
    assert kv.errors(reset=True) == DEVERR_PAGE
    t = kv.table.cpu()
    flat = kv.pages.view(-1, cfg.record_elems)
    rows = []
    for r, n in enumerate([60, 70, 80]):
        pos = [(0 if p < 50 else r, p) for p in range(n)]
        idx = [row_of(t, x, p, 16, 0) for x, p in pos if (x, p // 16) not in ((0, 1), (1, 4))]
        rows.append(flat[torch.tensor(idx, device=DEV)])
    want, bound, _ = ref.attention(cfg, rows + [flat[:0]] * 2, q, cfg.default_scale, [0] * 5)
    assert bool(((out.double() - want).abs() <= bound).all())
    assert torch.count_nonzero(w[1, 0, 64:70]) == 0 and bool((w[1, 0, 50:64] > 0).all())


@pytest.mark.parametrize("cfg", [gqa(6), mla(6), gqa(6, 4, 2, 80)], ids=["gqa", "mla", "any"])
def test_in_a_graph_on_streams_and_again(cfg):
    """A captured call reads lengths, groups and prefixes anew at each replay; equal calls give equal bits, on several streams at once."""
    groups, prefix, lens = [0, 4], [150], [170, 230, 300, 151, 40, 0]
    kv, q, out, acc = check(cfg, groups, prefix, lens, lists=1, slack=50)
    gt, pt = torch.tensor(groups, dtype=torch.int32, device=DEV), torch.tensor(prefix, device=DEV)
    lt = torch.tensor(lens, device=DEV)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [kv.prefix_attn(q, lt, groups=gt, prefix=pt, stream=s) for _ in range(5) for s in streams]
    assert kv.errors() == 0 and all(ref.same(x, out) for x in got)
    w = torch.rand(acc.shape, generator=gen(6), device=DEV)
    graph = torch.cuda.CUDAGraph()
    to = torch.zeros_like(out)
    with torch.cuda.graph(graph):
        kv.prefix_attn(q, lt, groups=gt, prefix=pt, weights=w, out=to)
    graph.replay()
    assert kv.errors() == 0 and ref.same(to, out) and ref.same(w, acc)
    for g2, p2, l2 in (([1, 6], [30], [100, 300, 31, 30, 200, 290]), ([0, 1], [20], [20, 1, 0, 0, 3, 333])):
        gt.copy_(torch.tensor(g2)), pt.copy_(torch.tensor(p2)), lt.copy_(torch.tensor(l2))
        w.copy_(torch.rand(w.shape, generator=gen(6), device=DEV))
        graph.replay()
        _, _, now, a2 = check(cfg, g2, p2, l2, kv=kv, q=q, lists=1, slack=350 - max(l2))
        assert ref.same(to, now) and ref.same(w, a2)


def test_refusals():
    kv = make_cache(gqa(2), 64, 16, 0)
    q = torch.zeros((2, 32, 128), dtype=torch.bfloat16, device=DEV)
    lens, w = torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros((2, 8, 64), device=DEV)
    groups, prefix = torch.tensor([0, 2], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    for kind, args, more in [
        (ValueError, (q[:, :16], lens), {}), (TypeError, (q.float(), lens), {}), (ValueError, (q.cpu(), lens), {}), (TypeError, (q, lens.int()), {}),
        (ValueError, (q, lens), dict(groups=groups)), (ValueError, (q, lens), dict(prefix=prefix)),
        (ValueError, (q, lens), dict(groups=groups, prefix=torch.zeros(3, dtype=torch.int64, device=DEV))),
        (ValueError, (q, lens), dict(groups=groups[:1], prefix=prefix)), (TypeError, (q, lens), dict(groups=groups.long(), prefix=prefix)),
        (TypeError, (q, lens), dict(weights=w.double())), (ValueError, (q, lens), dict(weights=w[:, :3])), (ValueError, (q, lens), dict(weights=w[0])),
        (ValueError, (q, lens), dict(weights=w, decay=float("nan"))), (ValueError, (q, lens), dict(scale=float("inf"))),
        (ValueError, (q, lens), dict(out=q[:1])), (HsError, (q, lens), dict(out=q)),
    ]:
        with pytest.raises(kind):
            kv.prefix_attn(*args, **more)
    assert kv.errors() == 0


@pytest.mark.parametrize("cfg,shared", [(gqa(4, 8, 2, 64), 40), (gqa(4), 0), (mla(4), 40), (gqa(4, 4, 2, 80), 33)], ids=["gqa64", "gqa", "mla", "any"])
def test_a_decode_loop_of_all_of_them(cfg, shared):
    """Append with norms, attend over the shared prefix and sum up weights, evict when a request is over its budget; each step
    against the 64-bit forms on what the cache holds."""
    R, Hq, Hk, D, Dv = cfg.num_requests, cfg.num_q_heads, cfg.num_kv_heads, cfg.head_dim_qk, cfg.head_dim_v
    latent = cfg.layout == 0
    page, budget, slack = 16, 70, 6
    kv = make_cache(cfg, budget + slack, page, 3)
    first = shared // page * page  # whole pages are in all tables
    for r in range(1, R):
        kv.table[r, : first // page] = kv.table[0, : first // page]
    lens = [shared] + [shared + 3 * r for r in range(1, R)]
    lt = torch.tensor(lens, dtype=torch.int64, device=DEV)
    seen = lt.clone()  # positions so far, evicted ones among them
    groups, prefix = torch.tensor([0, R], dtype=torch.int32, device=DEV), torch.tensor([shared], device=DEV)
    acc = torch.zeros((R, Hk, kv._kv.max_pages * page), device=DEV)
    cu = torch.arange(R + 1, dtype=torch.int32, device=DEV)
    rot = 16 if D == 80 else 64
    rope = RopeTable(rot, axes=[j % 2 for j in range(rot // 2)])
    inv = [10000.0 ** (-2 * j / rot) for j in range(rot // 2)]
    kw = 1 + 0.2 * torch.randn(Dv if latent else D, generator=gen(1), device=DEV)
    qw = None if latent else 1 + 0.2 * torch.randn(D, generator=gen(2), device=DEV)
    for step in range(20):
        k = torch.randn((R, Hk, D), generator=gen(100 + step), device=DEV).to(torch.bfloat16)
        v = None if latent else torch.randn((R, Hk, Dv), generator=gen(200 + step), device=DEV).to(torch.bfloat16)
        q = torch.randn((R, Hq, D), generator=gen(300 + step), device=DEV).to(torch.bfloat16)
        pos = torch.stack([seen, seen // 3], dim=1).contiguous()
        qr = kv.append(k, v, cu, lt, rope=rope, rope_pos=pos, q=q, k_weight=kw, q_weight=qw)
        off = D - rot if latent else 0
        x = ref.normed(k if not latent else k[..., :Dv], kw, 1e-6)
        want, bound = ref.turned(torch.cat([x, k[..., Dv:].double()], dim=-1) if latent else x, pos.tolist(), [j % 2 for j in range(rot // 2)], inv, off, False,
                                 Dv if latent else D)
        t = kv.table.cpu()
        rec = kv.pages.view(-1, cfg.record_elems)[[row_of(t, r, n, page, 0) for r, n in enumerate(lt.tolist())]].view(R, Hk, -1)[..., :D]
        assert bool(((rec.double() - want).abs() <= bound).all())
        lt += 1
        seen += 1
        lead, pre = shared_of(R, [0, R], [shared])
        before = acc.clone()
        out = kv.prefix_attn(qr, lt, groups=groups, prefix=prefix, weights=acc, decay=0.9)
        n = lt.tolist()
        want, bound, weights = ref.attention(cfg, rows_of(kv, lead, pre, n), qr, cfg.default_scale, [x - shared for x in n])
        assert bool(((out.double() - want).abs() <= bound).all())
        for r in range(R):
            w = weights[r].unflatten(1, (Hk, Hq // Hk)).sum(dim=2)
            new = 0.9 * before[r, :, shared:n[r]].double() + w[0]
            assert bool(((acc[r, :, shared:n[r]].double() - new).abs() <= w[1] + (Hq // Hk + 3) * U_FP32 * (2 * new + 1e-30)).all())
        cut = shared + 12 if step % slack == slack - 1 else 10**6
        if cut < 10**6:
            want, wout, wlens = ref.evict(kv.pages.cpu(), t, 0, acc.cpu(), acc.cpu(), n, cut, [shared] * R, 4)
            kv.evict(lt, acc, cut, first=shared, recent=4, lens_out=lt)
            assert lt.tolist() == wlens and ref.same(acc.cpu(), wout) and ref.same(kv.pages.cpu(), want)
    assert kv.errors() == 0
