"""The speculative-decoding operators on the GPU: rotate-and-append, tree attention (paged cache and pool),
keeping the accepted path; each against a plain 64-bit form, and together."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import spec_ref as ref
from hierarchical_kv_cache_02_gb300 import (DEVERR_APPEND, DEVERR_LOC, DEVERR_PAGE, LAYOUT_GQA, LAYOUT_MLA, HsConfig,
                                            HsError, HsPool, PagedKV, RopeTable, inputs, tree_mask)

DEV = "cuda:0"


def gqa(R, Hq=32, Hkv=8, D=128, Dv=None):
    return HsConfig(num_requests=R, num_layers=1, capacity=64, layout=LAYOUT_GQA, num_q_heads=Hq, num_kv_heads=Hkv,
                    head_dim_qk=D, head_dim_v=Dv or D, top_k=8, buffer_slots=16)


def mla(R, Hq=64, D=576, Dv=512):
    return HsConfig(num_requests=R, num_layers=1, capacity=64, layout=LAYOUT_MLA, num_q_heads=Hq, num_kv_heads=1,
                    head_dim_qk=D, head_dim_v=Dv, top_k=8, buffer_slots=16)


def randn(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def make_cache(cfg, most, page, seed, table=True, spare=3):
    """Random pages (some in no table) and a shuffled table for `most` positions a request."""
    R, each = cfg.num_requests, max(1, -(-most // page))
    n = R * each + (spare if table else 0)
    pages = randn((n, page, cfg.record_elems), seed)
    t = None
    if table:
        g = torch.Generator().manual_seed(seed)
        t = torch.randperm(n, generator=g)[: R * each].to(torch.int32).view(R, each).to(DEV)
    return PagedKV(cfg, pages, t)


def flat_rows(kv, r, positions):
    page, each = kv.pages.shape[1], kv._kv.max_pages
    table = kv.table.cpu() if kv.table is not None else None
    idx = [ref.row_of(table, r, int(p), page, each) for p in positions]
    return kv.pages.view(-1, kv.cfg.record_elems)[torch.tensor(idx, dtype=torch.int64, device=DEV)]


def random_tree(R, T, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.stack([torch.tensor([-1] + [int(torch.randint(-1, j, (1,), generator=g)) for j in range(1, T)])
                        for _ in range(R)])


def check_tree(cfg, kv, lens, T, mask, locs=None, nodes=None, seed=0, q=None, scale=None, only=None):
    R = cfg.num_requests
    if q is None:
        q = randn((R, T, cfg.num_q_heads, cfg.head_dim_qk), seed + 77)
    out = torch.full((R, T, cfg.num_q_heads, cfg.head_dim_v), 7.0, dtype=torch.bfloat16, device=DEV)
    before = out.clone()
    lt = torch.tensor(lens, dtype=torch.int64, device=DEV)
    nt = None if nodes is None else torch.tensor(nodes, dtype=torch.int32, device=DEV)
    got = kv.tree_attn(q, lt, mask.to(DEV), locs=locs, nodes=nt, out=out, scale=scale)
    assert got is out and kv.errors() == 0
    nn = nodes or [T] * R
    ctx = [flat_rows(kv, r, [p for p in (locs[r].tolist() if locs is not None else range(lens[r])) if p >= 0])
           for r in range(R)]
    node = [flat_rows(kv, r, range(lens[r], lens[r] + nn[r])) for r in range(R)]
    want, bound = ref.tree(cfg, ctx, node, q, mask.tolist(), nn, cfg.default_scale if scale is None else scale,
                           only=only)
    ref.assert_tree(out, want, bound, nn, before)
    return q, out


# (config of R requests, nodes, context lengths, page tokens)
TREES = [
    pytest.param(lambda: gqa(3), 4, [0, 1, 130], 16, id="gqa-short"),
    pytest.param(lambda: gqa(2), 1, [127, 128], 64, id="gqa-one-node"),
    pytest.param(lambda: gqa(2), 8, [1000, 257], 64, id="gqa-8"),
    pytest.param(lambda: gqa(1, 8, 2), 64, [300], 7, id="gqa-64-nodes-odd-pages"),
    pytest.param(lambda: gqa(2, 4, 2), 130, [129, 3], 1, id="gqa-130-nodes-pages-of-one"),
    pytest.param(lambda: gqa(1, 16, 1), 256, [515], 32, id="gqa-256-nodes"),
    pytest.param(lambda: gqa(2, 10, 2), 9, [400, 63], 100, id="gqa-group-of-5"),
    pytest.param(lambda: gqa(2, 7, 1, 64), 33, [77, 511], 16, id="gqa-64-dims-group-of-7"),
    pytest.param(lambda: gqa(2, 8, 8, 64), 5, [640, 12], 128, id="gqa-64-dims-ungrouped"),
    pytest.param(lambda: gqa(1, 40, 2), 3, [200], 16, id="gqa-group-of-20"),
    pytest.param(lambda: gqa(1, 130, 1), 2, [50], 16, id="gqa-group-of-130"),
    pytest.param(lambda: gqa(2, 4, 2, 192, 128), 6, [90, 33], 16, id="gqa-192-128"),
    pytest.param(lambda: gqa(2, 4, 2, 80), 6, [90, 33], 16, id="gqa-80"),
    pytest.param(lambda: gqa(1, 2, 1, 8), 3, [40], 16, id="gqa-8-dims"),
    pytest.param(lambda: gqa(1, 2, 1, 576), 3, [40], 16, id="gqa-576-dims"),
    pytest.param(lambda: mla(3), 4, [0, 1, 130], 16, id="mla-short"),
    pytest.param(lambda: mla(2), 1, [127, 64], 64, id="mla-one-node"),
    pytest.param(lambda: mla(2), 7, [700, 65], 64, id="mla-7"),
    pytest.param(lambda: mla(1, 128), 3, [200], 5, id="mla-128-heads"),
    pytest.param(lambda: mla(1, 16), 9, [300], 64, id="mla-16-heads"),
    pytest.param(lambda: mla(1, 40), 66, [90], 32, id="mla-40-heads-66-nodes"),
    pytest.param(lambda: mla(1, 130), 2, [90], 32, id="mla-130-heads"),
    pytest.param(lambda: mla(1, 4, 128, 64), 3, [90], 32, id="latent-128-64"),
]


@pytest.mark.parametrize("cfg,T,lens,page", TREES)
@pytest.mark.parametrize("table", [True, False])
def test_tree_over_a_dense_context(cfg, T, lens, page, table):
    cfg = cfg()
    kv = make_cache(cfg, max(lens) + T, page, seed=T + sum(lens), table=table)
    check_tree(cfg, kv, lens, T, tree_mask(random_tree(cfg.num_requests, T, seed=T)), seed=T)


@pytest.mark.parametrize("cfg,T,most", [(gqa(5), 7, 9000), (gqa(5), 70, 5000), (gqa(5, 40, 8), 77, 3000), (gqa(40, 2, 2, 64), 1, 700),
                                        (gqa(5, 32, 8, 64), 40, 6000), (gqa(300, 4, 2), 2, 200), (gqa(700, 2, 1), 2, 90),
                                        (mla(5), 3, 9000), (mla(60), 2, 300)])
@pytest.mark.parametrize("listed", [False, True])
def test_tree_with_many_tiles_and_requests_a_worker(cfg, T, most, listed):
    """Workers that walk through many tiles, several items and many requests, empty ones among them; every
    (request, node, head) is compared for a sample of them."""
    R, Hq = cfg.num_requests, cfg.num_q_heads
    g = torch.Generator().manual_seed(T)
    lens = [int(x) for x in torch.randint(0, most, (R,), generator=g)]
    lens[0] = most
    nodes = [T if r % 3 else int(torch.randint(0, T + 1, (1,), generator=g)) for r in range(R)]
    nodes[0] = T
    kv = make_cache(cfg, most + T, 16, seed=T)
    locs = None
    if listed:
        k = min(most, 1500)
        locs = torch.full((R, k), -1, dtype=torch.int32)
        for r in range(R):
            p = torch.randperm(lens[r] + 1, generator=g)[:k] if r % 4 else torch.arange(0)
            locs[r, :len(p)] = p.to(torch.int32)
        locs = locs.to(DEV)
    pick = torch.randint(0, 10**9, (150, 3), generator=g).tolist()
    only = {(a % R, b % T, c % Hq) for a, b, c in pick} | {(0, T - 1, Hq - 1), (R - 1, 0, 0)}
    check_tree(cfg, kv, lens, T, tree_mask(random_tree(R, T, seed=T)), locs=locs, nodes=nodes, seed=T, only=only)


@pytest.mark.parametrize("cfg,T,k", [(gqa(3), 8, 300), (gqa(2, 14, 2), 19, 1), (gqa(2, 8, 8, 64), 3, 129),
                                     (mla(3), 5, 300), (mla(2, 16), 2, 64), (gqa(2, 4, 2, 80), 3, 77)])
def test_tree_over_a_list_of_positions(cfg, T, k):
    """Lists in random order with padding anywhere, a list of nothing but padding, drafts behind lens."""
    R, rows = cfg.num_requests, 400
    kv = make_cache(cfg, rows + T, 16, seed=k)
    g = torch.Generator().manual_seed(k)
    locs = torch.stack([torch.randperm(rows, generator=g)[:k] for _ in range(R)]).to(torch.int32)
    locs[0, ::3] = -1
    locs[1] = -1
    check_tree(cfg, kv, [rows - 7 * r for r in range(R)], T, tree_mask(random_tree(R, T, seed=k)), locs=locs.to(DEV),
               seed=k)


@pytest.mark.parametrize("cfg", [gqa(4), gqa(4, 4, 2, 80), mla(4)], ids=["gqa", "any", "mla"])
@pytest.mark.parametrize("T", [6, 70])
def test_masks_of_any_pattern_and_nodes_in_use(cfg, T):
    """Random masks that are no tree, nodes that see nothing (zeros where the context is empty too), fewer
    nodes in use than the call has (none at all for one request): the rows behind stay as they were."""
    R, words = 4, (T + 63) // 64
    lens, nodes = [0, 50, 300, 20], [T, T - 2, 0, 1]
    kv = make_cache(cfg, max(lens) + T, 16, seed=5)
    g = torch.Generator().manual_seed(T)
    mask = torch.randint(-(2**63), 2**63 - 1, (R, T, words), generator=g, dtype=torch.int64)
    mask[:, 2] = 0
    mask[0, 0] = 0
    _, out = check_tree(cfg, kv, lens, T, mask, nodes=nodes)
    assert torch.count_nonzero(out[0, 0]) == 0 and torch.count_nonzero(out[0, 2]) == 0


@pytest.mark.parametrize("cfg,T", [(gqa(3), 4), (gqa(3), 70), (gqa(3, 8, 2, 64), 1), (gqa(3, 4, 2, 80), 2), (mla(3), 4), (gqa(40), 2),
                                   (mla(40), 1)])
def test_no_nodes_at_all(cfg, T):
    """Nothing to do: every output row stays as it was, and the call after it works."""
    R = cfg.num_requests
    kv = make_cache(cfg, 64 + T, 16, seed=T)
    mask = tree_mask(random_tree(R, T, seed=1))
    check_tree(cfg, kv, [60] * R, T, mask, nodes=[0] * R)
    check_tree(cfg, kv, [0] * R, T, mask, nodes=[0] * (R - 1) + [1])


@pytest.mark.parametrize("cfg", [gqa(2), gqa(2, 8, 2, 64), gqa(2, 4, 2, 80), mla(2), mla(2, 16)],
                         ids=["gqa", "gqa64", "any", "mla", "mla16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_node_does_not_see_has_no_influence(cfg, bad):
    """Two branches, one of them of NaN or infinite records; every row that no list names and every row
    behind the drafts as well: the other branch's outputs are those of a clean cache, bit for bit."""
    R, T, rows = 2, 12, 200
    kv = make_cache(cfg, rows + T + 20, 16, seed=3)
    parents = torch.tensor([[-1] + [max(-1, j - 2) for j in range(1, T)]] * R)  # even nodes and odd nodes
    mask = tree_mask(parents)
    locs = torch.arange(0, 2 * 90, 2, dtype=torch.int32).repeat(R, 1)
    lens = [rows, rows - 3]
    q, clean = check_tree(cfg, kv, lens, T, mask, locs=locs.to(DEV))
    flat = kv.pages.view(-1, cfg.record_elems)
    table, page = kv.table.cpu(), kv.pages.shape[1]
    good = [ref.row_of(table, r, p, page, 0) for r in range(R) for p in list(range(0, 180, 2)) +
            [lens[r] + j for j in range(0, T, 2)]]
    sick = torch.ones(flat.shape[0], dtype=torch.bool, device=DEV)
    sick[torch.tensor(good, device=DEV)] = False
    flat[sick] = bad
    out = torch.empty_like(clean)
    kv.tree_attn(q, torch.tensor(lens, dtype=torch.int64, device=DEV), mask.to(DEV), locs=locs.to(DEV), out=out)
    assert torch.equal(out[:, 0::2], clean[:, 0::2])
    assert not bool(torch.isfinite(out[:, 1::2]).any())


@pytest.mark.parametrize("cfg,dim", [(gqa(1), 3), (gqa(1), 127), (gqa(1, 8, 2, 64), 40), (gqa(1, 4, 2, 80), 79), (mla(1), 5),
                                     (mla(1), 300), (mla(1), 511), (mla(1), 570)])
@pytest.mark.parametrize("bad", [float("nan"), -float("inf")])
def test_one_bad_value_of_a_node_stays_where_it_is(cfg, dim, bad):
    """One infinite or NaN number in a node's value (shared latents: key and value at once), wherever it lies: rows that do
    not see the node keep their bits; of the others a GQA row loses this dim alone."""
    T, n = 11, 150
    lat = cfg.layout == LAYOUT_MLA
    kv = make_cache(cfg, n + T, 16, seed=dim)
    parents = torch.tensor([[-1] + [max(-1, j - 2) for j in range(1, T)]])  # even nodes and odd nodes
    mask = tree_mask(parents)
    q, clean = check_tree(cfg, kv, [n], T, mask, seed=dim)
    flat = kv.pages.view(-1, cfg.record_elems)
    sick = 4
    at = dim if lat else cfg.head_dim_qk + dim  # GQA: of the first KV head
    flat[ref.row_of(kv.table.cpu(), 0, n + sick, kv.pages.shape[1], 0), at] = bad
    out = kv.tree_attn(q, torch.tensor([n], dtype=torch.int64, device=DEV), mask.to(DEV))
    sees = torch.tensor([(mask[0, i, 0].item() >> sick) & 1 for i in range(T)], dtype=torch.bool)
    assert torch.equal(out[0, ~sees], clean[0, ~sees])
    if lat:
        assert not bool(torch.isfinite(out[0, sees]).any(dim=-1).all())
    else:
        G = cfg.num_q_heads // cfg.num_kv_heads
        hit = out[0, sees][:, :G]
        assert not bool(torch.isfinite(hit[..., dim]).any())
        same = clean[0, sees].clone()
        same[:, :G, dim] = hit[..., dim]
        assert torch.equal(out[0, sees].nan_to_num(nan=7.0), same.nan_to_num(nan=7.0))


def test_different_trees_at_once():
    """Trees of every kernel on three streams at once, again and again over long contexts: always the bits of the first
    call."""
    forms = [(gqa(3), 8, 9000, 64, False), (gqa(3), 70, 4000, 16, False), (mla(3), 5, 6000, 64, False), (mla(3), 2, 6000, 16, True),
             (gqa(3, 8, 2, 64), 5, 6000, 24, False), (gqa(3), 4, 6000, 64, True), (gqa(3, 4, 2, 80), 2, 300, 16, False)]
    calls, first = [], []
    for i, (cfg, T, n, page, listed) in enumerate(forms):
        R = cfg.num_requests
        kv = make_cache(cfg, n + T, page, seed=i)
        q = randn((R, T, cfg.num_q_heads, cfg.head_dim_qk), i)
        lens = torch.tensor([n, n // 3, n - 5], dtype=torch.int64, device=DEV)
        mask = tree_mask(random_tree(R, T, seed=i)).to(DEV)
        locs = None
        if listed:
            g = torch.Generator().manual_seed(i)
            locs = torch.stack([torch.randperm(n // 3, generator=g)[:1500] for _ in range(R)]).to(torch.int32).to(DEV)
        calls.append((kv, q, lens, mask, locs))
        first.append(kv.tree_attn(q, lens, mask, locs=locs))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for turn in range(8):
        outs = []
        for i in range(3 * len(calls)):
            kv, q, lens, mask, locs = calls[(i * 5 + turn) % len(calls)]
            outs.append(((i * 5 + turn) % len(calls), kv.tree_attn(q, lens, mask, locs=locs, stream=streams[i % 3])))
        torch.cuda.synchronize()
        for which, out in outs:
            assert torch.equal(out, first[which]), (turn, which)
    assert all(c[0].errors() == 0 for c in calls)


@pytest.mark.parametrize("cfg", [gqa(1), mla(1), gqa(1, 2, 1, 80)], ids=["gqa", "mla", "any"])
def test_scores_that_grow_and_fall_by_a_lot(cfg):
    """Sharp softmaxes whose maximum moves through the context, and all scores equal."""
    T, n = 3, 700
    kv = make_cache(cfg, n + T, 64, seed=9)
    q = randn((1, T, cfg.num_q_heads, cfg.head_dim_qk), 4)
    mask = tree_mask(random_tree(1, T, 1))
    check_tree(cfg, kv, [n], T, mask, q=q * 30)
    check_tree(cfg, kv, [n], T, mask, q=q * 0)
    check_tree(cfg, kv, [n], T, mask, q=q, scale=-0.25)
    check_tree(cfg, kv, [n], T, mask, q=q, scale=0.0)


def test_rows_beyond_32_bit_offsets():
    """A cache of more than 2^32 bytes (and more than 2^31 values) whose table names its last pages."""
    cfg = gqa(1)
    n = (1 << 32) // (cfg.record_bytes * 64) + 40
    pages = torch.zeros((n, 64, cfg.record_elems), dtype=torch.bfloat16, device=DEV)
    pages[n - 8:] = randn((8, 64, cfg.record_elems), 1)
    table = torch.arange(n - 1, n - 9, -1, dtype=torch.int32, device=DEV).view(1, 8)
    kv = PagedKV(cfg, pages, table)
    check_tree(cfg, kv, [400], 8, tree_mask(random_tree(1, 8, 1)))
    k, v = randn((5, 8, 128), 2), randn((5, 8, 128), 3)
    kv.append(k, v, torch.tensor([0, 5], dtype=torch.int32, device=DEV), torch.tensor([401], dtype=torch.int64, device=DEV))
    assert torch.equal(flat_rows(kv, 0, range(401, 406)).view(5, 8, 256), torch.cat([k, v], dim=2))
    kv.keep_path(torch.tensor([401], device=DEV), torch.tensor([[2, 4]], dtype=torch.int32, device=DEV),
                 torch.tensor([2], dtype=torch.int32, device=DEV))
    assert torch.equal(flat_rows(kv, 0, [401, 402]).view(2, 8, 256), torch.cat([k, v], dim=2)[[2, 4]])


def test_bad_positions_pages_lengths_and_counts_are_reported_and_not_seen():
    cfg = gqa(3)
    T = 2
    kv = make_cache(cfg, 60, 16, seed=1, spare=0)  # 4 pages a request: positions [0, 64)
    q = randn((3, T, 32, 128), 2)
    mask = tree_mask(torch.tensor([[-1, 0]] * 3)).to(DEV)

    def run(lens, locs=None, nodes=None):
        out = torch.zeros((3, T, 32, 128), dtype=torch.bfloat16, device=DEV)
        kv.tree_attn(q, torch.tensor(lens, dtype=torch.int64, device=DEV), mask, out=out,
                     locs=None if locs is None else torch.tensor(locs, dtype=torch.int32, device=DEV),
                     nodes=None if nodes is None else torch.tensor(nodes, dtype=torch.int32, device=DEV))
        return out

    good = run([10, 62, 5], locs=[[1, 2, 3]] * 3)
    assert kv.errors() == 0
    # listed positions outside the cache: as if they were padding
    out = run([10, 62, 5], locs=[[1, 2, 3], [1, 2, 3], [1, 2, 3]])
    assert torch.equal(out, good)
    a, b = run([10, 62, 5], locs=[[1, -1, 3]] * 3), run([10, 62, 5], locs=[[1, 64, 3], [1, -2, 3], [1, 2**31 - 1, 3]])
    assert torch.equal(a, b) and kv.errors(reset=True) == DEVERR_LOC
    # a context longer than the cache: what there is of it; no node fits behind it
    want = run([64, 3, 3], nodes=[T, T, T])
    assert kv.errors(reset=True) == DEVERR_LOC
    assert torch.equal(run([2**40, 3, 3])[0], want[0]) and kv.errors(reset=True) == DEVERR_LOC
    # a negative length: no context (its nodes' records lie before the cache); node counts out of range
    out = run([-1, 3, 3], nodes=[1, 3, -1])
    assert kv.errors(reset=True) == DEVERR_LOC
    assert torch.count_nonzero(out[0]) == 0 and torch.count_nonzero(out[2]) == 0
    assert torch.equal(out[1], run([3, 3, 3])[1]) and kv.errors() == 0
    # a table entry that is no page
    kv.table[1, 0] = kv.pages.shape[0]
    kv.table[2, 0] = -5
    out = run([10, 16, 17])
    assert kv.errors(reset=True) == DEVERR_PAGE
    assert bool(torch.isfinite(out).all()) and torch.equal(out[0], run([10, 0, 0])[0])
    kv.errors(reset=True)
    k = randn((3, 8, 128), 3)
    before = kv.pages.clone()
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    kv.append(k, k, cu, torch.tensor([64, 3, -1], dtype=torch.int64, device=DEV))
    assert kv.errors(reset=True) == DEVERR_APPEND | DEVERR_PAGE and torch.equal(kv.pages, before)
    kv.keep_path(torch.tensor([60, 3, 40], device=DEV), torch.tensor([[4, 0], [2, 3], [-1, 0]], dtype=torch.int32, device=DEV),
                 torch.tensor([2, 2, 3], dtype=torch.int32, device=DEV))
    assert kv.errors(reset=True) == DEVERR_LOC | DEVERR_PAGE and torch.equal(kv.pages, before)


# ---- append ------------------------------------------------------------------------------------


def check_append(cfg, N, counts, starts, page, rope, inv_freq, interleaved, q_dim=0, rope_pos=None, off=None, lead=0):
    R, Hkv, dqk, dv = cfg.num_requests, cfg.num_kv_heads, cfg.head_dim_qk, cfg.head_dim_v
    lat = cfg.layout == LAYOUT_MLA
    kv = make_cache(cfg, max(s + c for s, c in zip(starts, counts)), page, seed=N)
    # one projection's views, with columns nobody asked for between them
    w = [cfg.num_q_heads * q_dim, Hkv * dqk, 0 if lat else Hkv * dv]
    flat = randn((N, sum(w) + 24), N + 1)
    q = flat[:, 8:8 + w[0]].unflatten(1, (cfg.num_q_heads, q_dim)) if q_dim else None
    k = flat[:, 16 + w[0]:16 + w[0] + w[1]].unflatten(1, (Hkv, dqk))
    v = None if lat else flat[:, 24 + w[0] + w[1]:].unflatten(1, (Hkv, dv))
    cum = [lead + sum(counts[:r]) for r in range(R + 1)]
    before = kv.pages.clone()
    q_out = torch.full((N, cfg.num_q_heads, q_dim), 3.0, dtype=torch.bfloat16, device=DEV) if q_dim else None
    rp = None if rope_pos is None else torch.tensor(rope_pos, dtype=torch.int64, device=DEV)
    kv.append(k, v, torch.tensor(cum, dtype=torch.int32, device=DEV), torch.tensor(starts, dtype=torch.int64, device=DEV),
              rope=rope, rope_pos=rp, q=q, q_out=q_out, rotary_offset=off)
    assert kv.errors() == 0
    if off is None:
        off = dqk - 2 * len(inv_freq) if lat and inv_freq else 0
    who = [(r, i) for r in range(R) for i in range(counts[r])]
    pos = [rope_pos[lead + x] if rope_pos is not None else starts[r] + i for x, (r, i) in enumerate(who)]
    live = slice(lead, lead + len(who))
    table = kv.table.cpu()
    rows = torch.tensor([ref.row_of(table, r, starts[r] + i, page, 0) for r, i in who], dtype=torch.int64, device=DEV)
    want = before.view(-1, cfg.record_elems).double()
    bound = torch.zeros_like(want)
    kk, kb = ref.rotated(k[live], pos, inv_freq, off, interleaved)
    if not lat:
        kk, kb = torch.cat([kk, v[live].double()], dim=2), torch.cat([kb, torch.zeros_like(v[live]).double()], dim=2)
    want[rows], bound[rows] = kk.flatten(1), kb.flatten(1)
    got = kv.pages.view(-1, cfg.record_elems).double()
    assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() - bound).max())
    if q_dim:
        qw, qb = ref.rotated(q[live], pos, inv_freq, off if q_dim == dqk else 0, interleaved)
        assert bool(((q_out[live].double() - qw).abs() <= qb).all())
        assert bool((q_out[:lead] == 3.0).all()) and bool((q_out[lead + len(who):] == 3.0).all())
    return kv


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("cfg,rd,q_dim,off", [
    (gqa(3), 128, 128, None), (gqa(3), 64, 128, 32), (gqa(3, 6, 2, 64), 16, 64, None), (gqa(3, 3, 1, 24, 40), 16, 16, 8),
    (mla(3), 64, 64, None), (mla(3, 5), 64, 576, None), (gqa(3, 2, 2, 576), 576, 0, None)])
def test_append_rotated(cfg, rd, q_dim, off, interleaved):
    """Ragged requests (one without a token), padding tokens before and behind them, far start positions."""
    inv = [10000.0 ** (-j / (rd // 2)) for j in range(rd // 2)]
    check_append(cfg, 23, [7, 0, 11], [5, 9, 37], 16, RopeTable(rd, interleaved=interleaved), inv, interleaved, q_dim=q_dim,
                 off=off, lead=2)


@pytest.mark.parametrize("N", [0, 1, 4, 5, 1030])
def test_append_token_counts(N):
    inv = [500000.0 ** (-j / 64) for j in range(64)]
    if N == 0:
        cfg = gqa(1)
        kv = make_cache(cfg, 10, 16, seed=1)
        before = kv.pages.clone()
        e = torch.empty((0, 8, 128), dtype=torch.bfloat16, device=DEV)
        kv.append(e, e, torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV))
        assert torch.equal(kv.pages, before)
        return
    check_append(gqa(2), N, [N - N // 3, N // 3], [0, 3], 7, RopeTable(128, theta=500000.0), inv, False, q_dim=128)


def test_append_far_and_negative_angles():
    """Angles of positions up to 2^40 and below zero, given apart from where the records go."""
    inv = [1.0, 0.5, 2.0**-20, 1e-9, 3.0, 100.0, 0.0, 1.0 / 3]
    pos = [0, 1, 131071, 2**31 - 1, 2**31, 2**40 - 1, -1, -(2**33)]
    check_append(gqa(1, 4, 2, 64), 8, [8], [0], 16, RopeTable(16, inv_freq=inv), inv, False, q_dim=64, rope_pos=pos)


def test_append_without_rotation_copies_bits():
    check_append(gqa(2), 9, [4, 5], [0, 100], 16, None, [], False, q_dim=128)
    check_append(mla(2), 9, [4, 5], [0, 100], 16, None, [], False)


def test_append_in_place_query_and_special_values():
    """Queries rotated in place equal those rotated into another tensor; infinities and NaN of one token
    stay with it."""
    cfg = gqa(1)
    kv = make_cache(cfg, 40, 16, seed=2)
    q, k = randn((6, 32, 128), 1), randn((6, 8, 128), 2)
    q[3] = float("nan")
    k[3, 0, 0] = float("inf")
    cu, start = torch.tensor([0, 6], dtype=torch.int32, device=DEV), torch.tensor([20], dtype=torch.int64, device=DEV)
    rope = RopeTable(128)
    a = kv.append(k, k, cu, start, rope=rope, q=q)
    b = q.clone()
    assert kv.append(k, k, cu, start, rope=rope, q=b, q_out=b) is b
    ok = [0, 1, 2, 4, 5]
    assert torch.equal(a[ok], b[ok]) and bool(torch.isfinite(a[ok]).all()) and bool(a[3].isnan().all())
    rows = flat_rows(kv, 0, range(20, 26)).view(6, 8, 256)
    assert bool(torch.isfinite(rows[ok]).all()) and not bool(torch.isfinite(rows[3, 0, 0]))
    assert bool(torch.isfinite(rows[3, 1:]).all())


# ---- keep path ---------------------------------------------------------------------------------


@pytest.mark.parametrize("cfg,page", [(gqa(5), 16), (mla(5), 3), (gqa(5, 2, 1, 8), 64)])
def test_keep_path(cfg, page):
    T, P = 40, 20
    kv = make_cache(cfg, 100 + T, page, seed=page)
    g = torch.Generator().manual_seed(page)
    path = torch.zeros((5, P), dtype=torch.int32)
    counts = [0, 1, 9, 20, 20]
    for r, c in enumerate(counts):
        path[r, :c] = torch.sort(torch.randperm(T, generator=g)[:c]).values.to(torch.int32)
    path[4] = torch.arange(P)  # a chain accepted whole: nothing moves
    path[3] = torch.arange(P) + 1  # every record one place up
    lens = [0, 7, 31, 100, 64]
    want = kv.pages.clone().view(-1, cfg.record_elems)
    old, table = want.clone(), kv.table.cpu()
    for r, c in enumerate(counts):
        for i in range(c):
            want[ref.row_of(table, r, lens[r] + i, page, 0)] = old[ref.row_of(table, r, lens[r] + int(path[r, i]), page, 0)]
    kv.keep_path(torch.tensor(lens, device=DEV), path.to(DEV), torch.tensor(counts, dtype=torch.int32, device=DEV))
    assert kv.errors() == 0 and torch.equal(kv.pages.view(-1, cfg.record_elems), want)


# ---- together ----------------------------------------------------------------------------------


@pytest.mark.parametrize("cfg,rd", [(gqa(3), 128), (mla(3), 64), (gqa(3, 6, 2, 80), 80)], ids=["gqa", "mla", "any"])
def test_speculative_steps_equal_decoding_token_by_token(cfg, rd):
    """Three steps of append drafts -> tree attention -> keep path against a cache that only ever saw the
    accepted tokens, one at a time: the accepted nodes' outputs agree within the sum of both bounds, and
    the caches hold the same bits."""
    R, T, D = 3, 6, cfg.head_dim_qk
    rope = RopeTable(rd)
    spec, plain = make_cache(cfg, 80, 16, seed=8), make_cache(cfg, 80, 16, seed=9)
    lat = cfg.layout == LAYOUT_MLA
    parents = torch.tensor([[-1, 0, 0, 1, 2, -1]] * R)
    depth = torch.tensor([0, 1, 1, 2, 2, 0])
    mask = tree_mask(parents).to(DEV)
    paths = [[0, 2, 4], [0, 1], [5]]
    one = tree_mask(torch.tensor([[-1]] * R)).to(DEV)
    lens = torch.tensor([3, 0, 17], dtype=torch.int64, device=DEV)
    for cache in (spec, plain):  # the same context in both
        for r in range(R):
            for p in range(int(lens[r])):
                cache.pages.view(-1, cfg.record_elems)[ref.row_of(cache.table.cpu(), r, p, 16, 0)] = randn(
                    (cfg.record_elems,), 100 * r + p)
    for step in range(3):
        k, q = randn((R * T, cfg.num_kv_heads, D), 10 + step), randn((R * T, cfg.num_q_heads, D), 20 + step)
        v = None if lat else randn((R * T, cfg.num_kv_heads, cfg.head_dim_v), 30 + step)
        cu = torch.arange(0, R * T + 1, T, dtype=torch.int32, device=DEV)
        at = (lens[:, None] + depth.to(DEV)).reshape(-1).contiguous()
        qr = spec.append(k, v, cu, lens, rope=rope, rope_pos=at, q=q, q_out=torch.empty_like(q))
        out = spec.tree_attn(qr.view(R, T, cfg.num_q_heads, D), lens, mask)
        path = paths[step]
        P = torch.tensor([path] * R, dtype=torch.int32, device=DEV)
        count = torch.full((R,), len(path), dtype=torch.int32, device=DEV)
        spec.keep_path(lens, P, count)
        for i, node in enumerate(path):
            pick = torch.arange(R, device=DEV) * T + node
            q1 = plain.append(k[pick], None if lat else v[pick], torch.arange(R + 1, dtype=torch.int32, device=DEV), lens + i,
                              rope=rope, q=q[pick])
            o1 = plain.tree_attn(q1.view(R, 1, cfg.num_q_heads, D), lens + i, one)
            ctx = [flat_rows(plain, r, range(int(lens[r]) + i)) for r in range(R)]
            own = [flat_rows(plain, r, [int(lens[r]) + i]) for r in range(R)]
            want, bound = ref.tree(cfg, ctx, own, q1.view(R, 1, cfg.num_q_heads, D), one.tolist(), [1] * R, cfg.default_scale)
            ref.assert_tree(o1, want, bound, [1] * R)
            ref.assert_tree(out[:, node:node + 1], want, bound, [1] * R)
        lens = lens + len(path)
        for r in range(R):
            n = int(lens[r])
            assert torch.equal(flat_rows(spec, r, range(n)), flat_rows(plain, r, range(n))), (step, r)
    assert spec.errors() == 0 and plain.errors() == 0


@pytest.mark.parametrize("shape", ["gqa", "mla", "mla16"])
@pytest.mark.parametrize("device_pool", [False, True])
def test_tree_attention_over_a_pools_hot_buffers(shape, device_pool):
    """Resolve, then the tree attention over the published slots and drafts that were rotated by an append
    into a cache of their own: against the 64-bit form over the selected positions."""
    R, T, k, ctx, L = 3, 5, 96, 300, 2
    base = gqa(R) if shape == "gqa" else mla(R, 64 if shape == "mla" else 16)
    cfg = HsConfig(num_requests=R, num_layers=L, capacity=ctx, layout=base.layout, num_q_heads=base.num_q_heads,
                   num_kv_heads=base.num_kv_heads, head_dim_qk=base.head_dim_qk, head_dim_v=base.head_dim_v, top_k=k,
                   buffer_slots=128, device_pool_slots=128 * R * L if device_pool else 0)
    pool = HsPool(cfg)
    hist = inputs.normal_bf16((L, R, ctx, cfg.record_elems), seed=4)
    for l in range(L):
        for r in range(R):
            if device_pool:
                pool.reserve(r, ctx)
            pool.prefill(r, l, 0, hist[l, r])
    drafts = torch.zeros((R, T, cfg.record_elems), dtype=torch.bfloat16, device=DEV)
    dkv = PagedKV(cfg, drafts)
    mask = tree_mask(random_tree(R, T, 3)).to(DEV)
    g = torch.Generator().manual_seed(6)
    for step in range(2):
        for l in range(L):
            topk = torch.stack([torch.randperm(ctx, generator=g)[:k] for _ in range(R)]).to(torch.int32)
            topk[0, 5] = -1
            locs = pool.resolve(l, topk.to(DEV))
            kk = randn((R * T, cfg.num_kv_heads, cfg.head_dim_qk), 50 + step)
            vv = None if base.layout == LAYOUT_MLA else randn((R * T, cfg.num_kv_heads, cfg.head_dim_v), 60 + step)
            qq = randn((R * T, cfg.num_q_heads, cfg.head_dim_qk), 70 + l)
            q = dkv.append(kk, vv, torch.arange(0, R * T + 1, T, dtype=torch.int32, device=DEV),
                           torch.zeros(R, dtype=torch.int64, device=DEV), rope=RopeTable(64),
                           rope_pos=torch.arange(R * T, device=DEV) + ctx, q=qq).view(R, T, cfg.num_q_heads, -1)
            out = pool.tree_attn(l, q, locs, drafts, mask)
            rows = [hist[l, r][topk[r][topk[r] >= 0].long()].to(DEV) for r in range(R)]
            want, bound = ref.tree(cfg, rows, list(drafts), q, mask.tolist(), [T] * R, cfg.default_scale)
            ref.assert_tree(out, want, bound, [T] * R)
            # the pool's own attention still runs behind it
            pool.sparse_attn(l, q[:, 0].contiguous(), locs)
    assert pool.stats()["error_bits"] == 0
    bad = locs.clone()
    bad[1, 0], bad[1, 1] = 128, -7
    out = pool.tree_attn(1, q, bad, drafts, mask)
    none = locs.clone()
    none[1, 0] = none[1, 1] = -1
    assert pool.stats(reset=True)["error_bits"] == DEVERR_LOC
    assert torch.equal(out, pool.tree_attn(1, q, none, drafts, mask)) and pool.stats()["error_bits"] == 0
    pool.close()


def test_a_rotated_query_between_resolve_and_the_pools_attention():
    """The pool's attention may start before the whole resolve is done; a query rotated between the two has
    to be there all the same."""
    R, ctx, k = 16, 600, 512
    cfg = HsConfig(num_requests=R, num_layers=1, capacity=ctx, top_k=k, buffer_slots=512)
    pool = HsPool(cfg)
    hist = inputs.normal_bf16((R, ctx, cfg.record_elems), seed=4)
    for r in range(R):
        pool.prefill(r, 0, 0, hist[r])
    dkv = PagedKV(cfg, torch.zeros((R, 1, cfg.record_elems), dtype=torch.bfloat16, device=DEV))
    topk = torch.stack([torch.randperm(ctx)[:k] for _ in range(R)]).to(torch.int32).to(DEV)
    kk = randn((R, 8, 128), 1)
    cu, z = torch.arange(R + 1, dtype=torch.int32, device=DEV), torch.zeros(R, dtype=torch.int64, device=DEV)
    at = torch.arange(R, device=DEV) + ctx
    rope, q_out = RopeTable(128), torch.zeros((R, 32, 128), dtype=torch.bfloat16, device=DEV)
    for i in range(20):
        q = randn((R, 32, 128), 100 + i)
        torch.cuda.synchronize()
        locs = pool.resolve(0, topk)
        dkv.append(kk, kk, cu, z, rope=rope, rope_pos=at, q=q, q_out=q_out)
        got = pool.sparse_attn(0, q_out, locs)
        torch.cuda.synchronize()
        assert torch.equal(got, pool.sparse_attn(0, q_out, locs)), i
    pool.close()


def test_equal_calls_give_equal_bits_on_any_stream_and_in_graphs():
    """A step captured twice (two graphs, each with its own workspace), both replayed at once on two streams
    with new inputs in the captured tensors, equals eager calls bit for bit."""
    cfg, T, n = gqa(2), 8, 5000
    mask = tree_mask(random_tree(2, T, 1)).to(DEV)
    kvs = [make_cache(cfg, n + T, 64, seed=s) for s in (1, 2)]
    qs = [randn((2, T, 32, 128), s) for s in (3, 4)]
    ks = [randn((2 * T, 8, 128), s) for s in (5, 6)]
    lens = [torch.tensor([n, 900 + s], dtype=torch.int64, device=DEV) for s in (0, 1)]
    cu = torch.tensor([0, T, 2 * T], dtype=torch.int32, device=DEV)
    outs = [torch.zeros((2, T, 32, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    rope = RopeTable(128)
    path, count = torch.tensor([[1, 4], [0, 2]], dtype=torch.int32, device=DEV), torch.tensor([2, 1], dtype=torch.int32, device=DEV)

    def step(i, out):
        qr = kvs[i].append(ks[i], ks[i], cu, lens[i], rope=rope, q=qs[i].view(2 * T, 32, 128))
        kvs[i].tree_attn(qr.view(2, T, 32, 128), lens[i], mask, out=out)
        kvs[i].keep_path(lens[i], path, count)

    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        step(i, outs[i])
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            step(i, outs[i])
        graphs.append(g)
    for turn in range(3):
        for i in range(2):
            qs[i].copy_(randn((2, T, 32, 128), 40 + 2 * turn + i))
            ks[i].copy_(randn((2 * T, 8, 128), 60 + 2 * turn + i))
            lens[i].copy_(torch.tensor([n - 100 * turn, 64 * turn], device=DEV))
        start = [kv.pages.clone() for kv in kvs]
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        replayed, pages = [o.clone() for o in outs], [kv.pages.clone() for kv in kvs]
        for i in range(2):
            kvs[i].pages.copy_(start[i])
            torch.cuda.synchronize()
            other = torch.zeros_like(outs[i])
            for _ in range(3):
                step(i, other)
            torch.cuda.synchronize()
            assert torch.equal(other, replayed[i]) and torch.equal(kvs[i].pages, pages[i]), (turn, i)
            with torch.cuda.stream(streams[i]):  # the current stream
                a = kvs[i].tree_attn(qs[i], lens[i], mask)
            b = kvs[i].tree_attn(qs[i], lens[i], mask, stream=streams[1 - i])  # a given one
            torch.cuda.synchronize()
            assert torch.equal(a, b)


def test_refusals_on_tensors():
    cfg = gqa(2)
    kv = make_cache(cfg, 100, 16, seed=1)
    q = randn((2, 4, 32, 128), 1)
    lens = torch.tensor([3, 4], dtype=torch.int64, device=DEV)
    mask = tree_mask(random_tree(2, 4, 1)).to(DEV)
    k, cu = randn((6, 8, 128), 1), torch.tensor([0, 2, 6], dtype=torch.int32, device=DEV)
    rope = RopeTable(64)
    refused = (ValueError, TypeError, HsError)
    for call in [
        lambda: kv.tree_attn(q[0], lens, mask),
        lambda: kv.tree_attn(q.float(), lens, mask),
        lambda: kv.tree_attn(q.transpose(1, 2), lens, mask),
        lambda: kv.tree_attn(q, lens.int(), mask),
        lambda: kv.tree_attn(q, lens.cpu(), mask),
        lambda: kv.tree_attn(q, lens, mask[:, :3]),
        lambda: kv.tree_attn(q, lens, mask, locs=torch.zeros((2, 0), dtype=torch.int32, device=DEV)),
        lambda: kv.tree_attn(q, lens, mask, locs=torch.zeros((1, 3), dtype=torch.int32, device=DEV)),
        lambda: kv.tree_attn(q, lens, mask, nodes=torch.zeros((3,), dtype=torch.int32, device=DEV)),
        lambda: kv.tree_attn(q, lens, mask, out=torch.zeros((2, 4, 32, 128), device=DEV)),
        lambda: kv.tree_attn(q, lens, mask, scale=float("nan")),
        lambda: kv.tree_attn(randn((2, 257, 32, 128), 1), lens, torch.zeros((2, 257, 5), dtype=torch.int64, device=DEV)),
        lambda: kv.append(k, None, cu, lens),
        lambda: kv.append(k, k[:5], cu, lens),
        lambda: kv.append(k[:, :, ::2], k, cu, lens),
        lambda: kv.append(randn((6, 8 * 128 + 4), 1)[:, 4:].unflatten(1, (8, 128)), k, cu, lens),
        lambda: kv.append(k, k, cu[:2], lens),
        lambda: kv.append(k, k, cu.long(), lens),
        lambda: kv.append(k, k, cu, lens.int()),
        lambda: kv.append(k, k, cu, lens, rope=rope, rotary_offset=72),
        lambda: kv.append(k, k, cu, lens, rope=rope, rotary_offset=4),
        lambda: kv.append(k, k, cu, lens, rope=rope, rope_pos=lens),
        lambda: kv.append(k, k, cu, lens, rope=rope, q=randn((6, 32, 96), 1)),
        lambda: kv.append(k, k, cu, lens, q_out=randn((6, 32, 128), 1)),
        lambda: kv.append(k, k, cu, lens, q=randn((6, 32, 128), 1), q_out=randn((1, 32, 128), 1).expand(6, -1, -1)),
        lambda: kv.keep_path(lens, torch.zeros((2, 257), dtype=torch.int32, device=DEV), cu[:2].contiguous()),
        lambda: kv.keep_path(lens, torch.zeros((2, 3), dtype=torch.int64, device=DEV), cu[:2].contiguous()),
        lambda: kv.keep_path(lens, torch.zeros((2, 3), dtype=torch.int32, device=DEV), cu),
        lambda: PagedKV(cfg, torch.zeros((4, 16, 100), dtype=torch.bfloat16, device=DEV)),
        lambda: PagedKV(cfg, torch.zeros((5, 16, cfg.record_elems), dtype=torch.bfloat16, device=DEV)),
        lambda: PagedKV(cfg, torch.zeros((4, 16, cfg.record_elems), dtype=torch.bfloat16)),
        lambda: PagedKV(cfg, kv.pages, kv.table.long()),
        lambda: RopeTable(24),
        lambda: RopeTable(64, inv_freq=[1.0]),
        lambda: RopeTable(16, inv_freq=[float("inf")] * 8),
    ]:
        with pytest.raises(refused):
            call()
    fetching = HsConfig(num_requests=2, num_layers=1, capacity=64, top_k=8, buffer_slots=16, fetch_in_attention=1)
    pool = HsPool(fetching)
    with pytest.raises(HsError):
        pool.tree_attn(0, q, torch.zeros((2, 8), dtype=torch.int32, device=DEV), randn((2, 4, 2048), 1), mask)
    pool.close()
    assert kv.errors() == 0
