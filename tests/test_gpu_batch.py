"""The operators of a batch's decode step on the GPU: appends with norms and axes, eviction by weight; each against a
plain 64-bit form."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import batch_ref as ref
from hierarchical_kv_cache_02_gb300 import (DEVERR_APPEND, DEVERR_LOC, DEVERR_PAGE, LAYOUT_GQA, LAYOUT_MLA, HsConfig, HsError,
                                            PagedKV, RopeTable)
from spec_ref import row_of

DEV = "cuda:0"


def gqa(R, Hq=32, Hkv=8, D=128, Dv=None):
    return HsConfig(num_requests=R, num_layers=1, capacity=64, layout=LAYOUT_GQA, num_q_heads=Hq, num_kv_heads=Hkv,
                    head_dim_qk=D, head_dim_v=Dv or D, top_k=8, buffer_slots=16)


def mla(R, Hq=64, D=576, Dv=512):
    return HsConfig(num_requests=R, num_layers=1, capacity=64, layout=LAYOUT_MLA, num_q_heads=Hq, num_kv_heads=1,
                    head_dim_qk=D, head_dim_v=Dv, top_k=8, buffer_slots=16)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def make_cache(cfg, most, page, seed, table=True, spare=3):
    """Random pages (some in no table) and a shuffled table for `most` positions a request."""
    R, each = cfg.num_requests, max(1, -(-most // page))
    n = R * each + (spare if table else 0)
    pages = torch.randn((n, page, cfg.record_elems), generator=gen(seed), device=DEV).to(torch.bfloat16)
    t = None
    if table:
        t = torch.randperm(n, generator=torch.Generator().manual_seed(seed))[: R * each].to(torch.int32).view(R, each).to(DEV)
    return PagedKV(cfg, pages, t)


# ---- append with norms ---------------------------------------------------------------------------


def check_append(cfg, counts, page=16, rotary=64, off=None, interleaved=False, axes=1, kind=torch.bfloat16, per_head=False,
                 with_q=True, q_norm=True, k_norm=True, in_place=False, eps=1e-5, first=100, pad=(0, 0), seed=0, table=True, far=0):
    R, Hq, Hk, D = cfg.num_requests, cfg.num_q_heads, cfg.num_kv_heads, cfg.head_dim_qk
    latent = cfg.layout == LAYOUT_MLA
    Dv = cfg.head_dim_v
    N = sum(counts) + sum(pad)
    g = gen(seed + 1)
    kv = make_cache(cfg, first + max(counts) + 5, page, seed, table)
    before = kv.pages.clone()
    cu = [pad[0]]
    for c in counts:
        cu.append(cu[-1] + c)
    start = [first + 3 * r % 5 for r in range(R)]
    at = [(r, start[r] + i) for r, c in enumerate(counts) for i in range(c)]
    qd = rotary if latent else D
    flat = torch.randn((N, Hq * qd + Hk * D + (0 if latent else Hk * Dv) + 8), generator=g, device=DEV)
    flat = (flat * torch.logspace(-3, 3, N, device=DEV)[:, None]).to(torch.bfloat16)
    q = flat[:, : Hq * qd].unflatten(1, (Hq, qd))
    k = flat[:, Hq * qd : Hq * qd + Hk * D].unflatten(1, (Hk, D))
    v = None if latent else flat[:, Hq * qd + Hk * D : Hq * qd + Hk * (D + Dv)].unflatten(1, (Hk, Dv))
    q0, k0 = q.clone(), k.clone()
    dim = Dv if latent else D

    def weight(heads):
        return (1 + torch.randn((heads, dim) if per_head else (dim,), generator=g, device=DEV)).to(kind)

    kw, qw = weight(Hk) if k_norm else None, weight(Hq) if with_q and q_norm and not latent else None
    inv = [10000.0 ** (-2 * j / rotary) for j in range(rotary // 2)]
    axis = [j % axes for j in range(rotary // 2)]
    rope = RopeTable(rotary, inv_freq=inv, interleaved=interleaved, axes=axis if axes > 1 else None) if rotary else None
    pos = torch.randint(0, 1 << 20, (N, axes), generator=g, device=DEV) + far
    rope_pos = None if not far and axes == 1 else (pos if axes > 1 else pos[:, 0].contiguous())
    q_out = (q if in_place else torch.full((N, Hq, qd), 7.0, dtype=torch.bfloat16, device=DEV)) if with_q else None
    got = kv.append(k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), torch.tensor(start, dtype=torch.int64, device=DEV), rope=rope,
                    rope_pos=rope_pos, q=q if with_q else None, q_out=q_out, rotary_offset=off, q_weight=qw, k_weight=kw, eps=eps)
    assert kv.errors() == 0 and (got is q_out)
    live = slice(pad[0], N - pad[1])
    where = [[p] for _, p in at] if rope_pos is None else pos[live].tolist()
    koff = (D - rotary if latent else 0) if off is None else off
    x = k0[live].double()
    if kw is not None:
        x = torch.cat([ref.normed(k0[live][..., :dim], kw, eps), x[..., dim:]], dim=-1)
    want, bound = ref.turned(x, where, axis, inv if rotary else [], koff, interleaved, dim if kw is not None else 0)
    rows = [row_of(kv.table.cpu() if table else None, r, p, page, kv._kv.max_pages) for r, p in at]
    after = kv.pages.view(-1, cfg.record_elems)
    rec = after[rows].view(len(rows), Hk, -1)
    assert bool(((rec[..., :D].double() - want).abs() <= bound).all())
    if not latent:
        assert ref.same(rec[..., D:], v[live])
    rest = torch.ones(after.shape[0], dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert ref.same(after[rest], before.view(-1, cfg.record_elems)[rest])
    if with_q:
        x = q0[live].double() if qw is None else ref.normed(q0[live], qw, eps)
        want, bound = ref.turned(x, where, axis, inv if rotary else [], 0 if qd == rotary else koff, interleaved,
                                 dim if qw is not None else 0)
        assert bool(((q_out[live].double() - want).abs() <= bound).all())
        for s in (slice(0, pad[0]), slice(N - pad[1], N)):
            assert ref.same(q_out[s], q0[s] if in_place else torch.full_like(q0[s], 7.0))


@pytest.mark.parametrize("cfg,counts,more", [
    (gqa(1), [1], {}),
    (gqa(3), [5, 0, 9], dict(rotary=128)),
    (gqa(3), [5, 0, 9], dict(rotary=128, interleaved=True, kind=torch.float32)),
    (gqa(2, 40, 8), [7, 33], dict(rotary=32, off=96, per_head=True)),
    (gqa(2, 40, 8), [7, 33], dict(rotary=32, off=40, per_head=True, interleaved=True, kind=torch.float32)),
    (gqa(4, 28, 4, 64), [100, 1, 2, 600], dict(in_place=True, pad=(2, 3))),
    (gqa(4, 28, 4, 64), [1000, 1, 700, 600], dict(rotary=16, off=8, page=7)),
    (gqa(2, 6, 3, 80), [3, 4], dict(rotary=48, kind=torch.float32)),
    (gqa(2, 4, 2, 8), [3, 4], dict(rotary=0)),
    (gqa(2, 2, 1, 576), [3, 40], dict(rotary=576, kind=torch.float32, per_head=True)),
    (gqa(2, 2, 1, 576), [3, 40], dict(rotary=64, interleaved=True)),
    (gqa(2, 4, 2, 192, 128), [9, 9], dict(rotary=64, off=128)),
    (gqa(2, 4, 4, 64, 256), [9, 9], dict(rotary=64)),
    (gqa(2), [9, 12], dict(q_norm=False, table=False)),
    (gqa(2), [9, 12], dict(k_norm=False)),
    (gqa(2), [9, 12], dict(with_q=False)),
    (gqa(2), [4000, 3000], dict(rotary=128, page=64, pad=(1, 0))),
    (mla(3), [5, 0, 9], {}),
    (mla(3), [5, 100, 900], dict(interleaved=True, kind=torch.float32)),
    (mla(2, 16, 128, 64), [8, 9], dict(rotary=64)),
    (mla(2, 5, 96, 96), [8, 9], dict(rotary=32, off=0)),
    (mla(1, 130), [17], dict(rotary=64, per_head=True)),
    (gqa(2, 1024, 1, 16), [3, 2], dict(rotary=16)),
])
@pytest.mark.parametrize("axes,far", [(1, 0), (1, 1 << 33), (3, 0), (4, 1 << 33)])
def test_append_with_norms(cfg, counts, more, axes, far):
    if axes > 1 and more.get("rotary", 64) == 0:
        pytest.skip("nothing is rotated")
    check_append(cfg, counts, axes=axes, far=far, seed=len(counts) + axes, **more)


def test_a_table_with_axes_and_no_norms():
    check_append(gqa(3), [5, 0, 9], rotary=128, axes=3, q_norm=False, k_norm=False)
    check_append(mla(3), [5, 0, 9], axes=2, interleaved=True, k_norm=False)


def test_zeros_and_small_and_large_heads():
    """eps alone under the root; heads whose squares are near the smallest and largest 32-bit numbers."""
    cfg = gqa(1, 2, 1, 64)
    kv = make_cache(cfg, 8, 8, 0)
    x = torch.randn((4, 64), generator=gen(1), device=DEV)
    x = (x * torch.tensor([[0.0], [1e-20], [1e15], [1e-3]], device=DEV)).to(torch.bfloat16)[:, None]
    w = torch.ones(64, device=DEV)
    kv.append(x, torch.zeros_like(x), torch.tensor([0, 4], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV), k_weight=w,
              eps=1e-6)
    rows = [row_of(kv.table.cpu(), 0, p, 8, 1) for p in range(4)]
    got = kv.pages.view(-1, 128)[rows][:, :64].double()
    want, bound = ref.turned(ref.normed(x, w, 1e-6), [[0]] * 4, [], [], 0, False, 64)
    assert bool(((got - want[:, 0]).abs() <= bound[:, 0]).all()) and torch.count_nonzero(got[0]) == 0


def test_appends_report_bad_positions_and_pages():
    cfg = gqa(2, 4, 2, 64)
    kv = make_cache(cfg, 16, 8, 0)
    kv.table[1, 0] = 99
    before = kv.pages.clone()
    k = torch.randn((6, 2, 64), generator=gen(1), device=DEV).to(torch.bfloat16)
    q = torch.randn((6, 4, 64), generator=gen(2), device=DEV).to(torch.bfloat16)
    w = torch.ones(64, device=DEV)
    args = (k, k, torch.tensor([0, 3, 6], dtype=torch.int32, device=DEV))
    out = kv.append(*args, torch.tensor([15, 0], dtype=torch.int64, device=DEV), q=q, q_weight=w, k_weight=w)
    assert kv.errors(reset=True) == DEVERR_APPEND | DEVERR_PAGE
    want, bound = ref.turned(ref.normed(q, w, 1e-6), [[0]] * 6, [], [], 0, False, 64)
    assert bool(((out.double() - want).abs() <= bound).all())
    row = row_of(kv.table.cpu(), 0, 15, 8, 2)
    changed = (kv.pages != before).flatten(0, 1).any(dim=1)
    assert changed.nonzero().flatten().tolist() == [row]


# ---- eviction ------------------------------------------------------------------------------------


def check_evict(cfg, lens, keep, first=0, recent=0, heads=False, page=16, seed=0, table=True, weights=None, in_place=False, slack=0,
                tensor_first=None, cap=None):
    R, lists = cfg.num_requests, cfg.num_kv_heads if heads else 1
    kv = make_cache(cfg, max(lens) + slack, page, seed, table)
    cap = cap or max(1, max(lens)) + slack
    if weights is None:
        weights = torch.exp(2 * torch.randn((R, lists, cap), generator=gen(seed + 1), device=DEV))
        weights[torch.rand(weights.shape, generator=gen(seed + 2), device=DEV) < 0.2] = 0.0
    given = weights.clone()
    out = weights if in_place else torch.full_like(weights, 5.0)
    lt = torch.tensor(lens, dtype=torch.int64, device=DEV)
    f = first if tensor_first is None else torch.tensor(tensor_first, dtype=torch.int64, device=DEV)
    t = kv.table.cpu() if table else None
    want, wout, wlens = ref.evict(kv.pages.cpu(), t, kv._kv.max_pages, given.cpu(), out.cpu(), lens, keep,
                                  tensor_first or [first] * R, recent)
    got = kv.evict(lt, weights, keep, first=f, recent=recent, weights_out=None if in_place else out, lens_out=lt if in_place else None)
    assert kv.errors() == 0
    assert got.tolist() == wlens and (got is lt) == in_place
    assert ref.same(out.cpu(), wout)
    assert ref.same(kv.pages.cpu(), want)
    if not in_place:
        assert ref.same(weights, given)


@pytest.mark.parametrize("cfg,lens,keep,more", [
    (gqa(4), [0, 1, 30, 31], 30, {}),
    (gqa(3), [100, 64, 65], 64, dict(first=4, recent=10)),
    (gqa(3), [100, 64, 65], 64, dict(first=4, recent=60, heads=True)),
    (gqa(2), [1000, 700], 1, {}),
    (gqa(2), [1000, 700], 1, dict(recent=1)),
    (gqa(2), [1000, 700], 500, dict(first=500)),
    (gqa(2), [1000, 700], 699, dict(page=7)),
    (gqa(2, 8, 2, 64), [3000, 2049], 2048, dict(heads=True, first=16, recent=512)),
    (gqa(2, 8, 2, 64), [3000, 2049], 2048, dict(table=False, page=1)),
    (gqa(2, 4, 4, 8), [300, 200], 100, dict(heads=True)),
    (gqa(2, 4, 2, 80, 40), [300, 200], 100, dict(heads=True)),
    (gqa(40, 2, 1, 8), [17 * r % 90 for r in range(40)], 33, dict(recent=3)),
    (mla(2), [3000, 100], 1000, dict(first=4)),
    (mla(1), [257], 256, {}),
    (mla(20), [50 + r for r in range(20)], 60, dict(recent=8)),
    (mla(1, 2, 8, 8), [70000], 20000, dict(first=100, recent=1000)),
    (mla(2, 2, 8, 8), [70000, 49153], 49152, {}),
    (gqa(2, 4, 4, 8), [60000, 50000], 30001, dict(heads=True, slack=11)),
    (mla(1, 2, 8, 8), [9100], 4000, dict(page=2, recent=4)),
    (gqa(2, 2, 1, 8), [6000, 5000], 4500, dict(page=1, first=4200)),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(cfg, lens, keep, more, in_place):
    check_evict(cfg, lens, keep, seed=keep, in_place=in_place, **more)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_with_weights_of_every_kind(in_place):
    """Equal weights, zeros of both signs, negative ones, infinities and NaN; weights behind a length are not looked at."""
    nan, inf = float("nan"), float("inf")
    cfg = gqa(6, 4, 2, 64)
    w = torch.zeros((6, 2, 40), device=DEV)
    w[1] = 1.0
    w[2, :, ::3] = -0.0
    w[2, 1] = -torch.arange(40, device=DEV)
    w[3, 0, 5:20] = nan
    w[3, 1, 5:30] = nan
    w[3, :, 30:33] = inf
    w[4] = torch.tensor([-inf, inf, nan, -nan, 0.0, -0.0, 1.0, -1.0, 1e-45, -1e-45] * 4, device=DEV)
    w[5, :, 30:] = nan
    w[5, :, :30] = torch.randint(0, 3, (2, 30), generator=gen(0), device=DEV)
    check_evict(cfg, [40, 40, 40, 40, 40, 30], 17, first=2, recent=3, heads=True, weights=w, in_place=in_place, slack=0, cap=40)


def test_evict_with_a_first_of_each_request():
    check_evict(gqa(4), [100, 50, 90, 80], 40, recent=10, tensor_first=[0, 30, 17, 30])


def test_evict_leaves_bad_requests_alone():
    cfg = gqa(5, 4, 2, 64)
    kv = make_cache(cfg, 64, 16, 3)
    w = torch.rand((5, 2, 60), generator=gen(1), device=DEV)
    pages, w0 = kv.pages.clone(), w.clone()
    lens = torch.tensor([61, -1, 50, 1 << 40, 50], dtype=torch.int64, device=DEV)
    first = torch.tensor([0, 0, 31, 0, -1], dtype=torch.int64, device=DEV)
    out = torch.full_like(w, 3.0)
    new = kv.evict(lens, w, 40, first=first, recent=10, weights_out=out)
    assert kv.errors(reset=True) == DEVERR_LOC
    assert new.tolist() == lens.tolist() and ref.same(kv.pages, pages) and ref.same(w, w0) and bool((out == 3.0).all())
    kv.table[0, 3] = 1000
    kv.evict(torch.tensor([60, 0, 0, 0, 0], dtype=torch.int64, device=DEV), w, 40, recent=40)
    assert kv.errors(reset=True) == DEVERR_PAGE


def test_evict_in_a_graph_and_on_another_stream():
    """A captured call looks at the lengths and weights of each replay; two graphs share nothing."""
    cfg = gqa(3, 8, 2, 64)
    side = torch.cuda.Stream()
    kv = make_cache(cfg, 200, 16, 3)
    lens, w = torch.zeros(3, dtype=torch.int64, device=DEV), torch.zeros((3, 2, 200), device=DEV)
    new = torch.zeros_like(lens)
    for keep in (50, 20):  # two graphs of one pool
        graph = torch.cuda.CUDAGraph()
        kv.evict(lens, w, keep, lens_out=new, stream=side)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            kv.evict(lens, w, keep, lens_out=new)
        for n in ([200, 10, 100], [60, 60, 61]):
            kv.pages.copy_(torch.randn(kv.pages.shape, generator=gen(sum(n)), device=DEV))
            w.copy_(torch.rand(w.shape, generator=gen(keep), device=DEV))
            lens.copy_(torch.tensor(n))
            want, wout, wlens = ref.evict(kv.pages.cpu(), kv.table.cpu(), 0, w.cpu(), w.cpu(), n, keep, [0] * 3, 0)
            graph.replay()
            assert kv.errors() == 0 and new.tolist() == wlens and ref.same(w.cpu(), wout) and ref.same(kv.pages.cpu(), want)


# ---- refusals ------------------------------------------------------------------------------------


def test_refusals_of_appends():
    cfg = gqa(2)
    kv = make_cache(cfg, 64, 16, 0)
    k = torch.zeros((4, 8, 128), dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((4, 32, 128), dtype=torch.bfloat16, device=DEV)
    cu, start = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int64, device=DEV)
    w = torch.ones(128, device=DEV)
    rope = RopeTable(128, axes=[j % 2 for j in range(64)])
    for kind, more in [
        (TypeError, dict(k_weight=w.half())), (ValueError, dict(k_weight=w[:64].contiguous())), (ValueError, dict(k_weight=w.cpu())),
        (ValueError, dict(k_weight=torch.ones((32, 128), device=DEV))), (ValueError, dict(q=q, q_weight=torch.ones((8, 128), device=DEV))),
        (ValueError, dict(q_weight=w)), (ValueError, dict(k_weight=w, eps=0.0)), (ValueError, dict(k_weight=w, eps=float("nan"))),
        (ValueError, dict(k_weight=w, eps=float("inf"))), (ValueError, dict(k_weight=torch.ones(129, device=DEV)[1:])),
        (ValueError, dict(rope=rope)), (ValueError, dict(rope=rope, rope_pos=torch.zeros(4, dtype=torch.int64, device=DEV))),
        (ValueError, dict(rope=rope, rope_pos=torch.zeros((4, 3), dtype=torch.int64, device=DEV))),
        (ValueError, dict(rope=rope, q=q[..., :64], k_weight=w)),
    ]:
        with pytest.raises(kind):
            kv.append(k, k, cu, start, **more)
    latent = make_cache(mla(1), 64, 16, 0)
    with pytest.raises(ValueError):
        latent.append(torch.zeros((1, 576), dtype=torch.bfloat16, device=DEV), None, cu[:2].contiguous(), start[:1],
                      q=torch.zeros((1, 64, 576), dtype=torch.bfloat16, device=DEV), q_weight=torch.ones(512, device=DEV))
    for axes in ([0] * 63, [0.5] * 64, [-1] * 64, [4] * 64):
        with pytest.raises(ValueError):
            RopeTable(128, axes=axes)
    assert RopeTable(128, axes=[0] * 64).axis is None
    assert kv.errors() == 0


def test_refusals_of_evictions():
    kv = make_cache(gqa(2), 64, 16, 0)
    lens, w = torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros((2, 8, 64), device=DEV)
    for kind, args, more in [
        (ValueError, (lens, w, 0), {}), (ValueError, (lens, w, 10), dict(first=6, recent=5)), (ValueError, (lens, w, 10), dict(recent=-1)),
        (ValueError, (lens, w, 10), dict(first=-1)), (ValueError, (lens, w[:, :2], 10), {}), (ValueError, (lens, w[0], 10), {}),
        (TypeError, (lens, w.double(), 10), {}), (TypeError, (lens.int(), w, 10), {}), (ValueError, (lens, w, 1 << 31), {}),
        (ValueError, (lens, w, 10), dict(weights_out=w[:, :1])), (ValueError, (lens, w.transpose(0, 1), 10), {}),
        (TypeError, (lens, w, 10), dict(first=lens.int())), (ValueError, (lens, w.cpu(), 10), {}), (TypeError, (lens, w, 10), dict(lens_out=lens.int())),
    ]:
        with pytest.raises(kind):
            kv.evict(*args, **more)
    big = torch.zeros(2 * 8 * 64 + 8, device=DEV)
    with pytest.raises(HsError):
        kv.evict(lens, big[:1024].view(2, 8, 64), 10, weights_out=big[8:].view(2, 8, 64))
    assert kv.errors() == 0
