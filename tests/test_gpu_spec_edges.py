"""Edges of the speculative-decoding operators on the GPU that the operators' own tests leave out."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import spec_ref as ref
from hierarchical_kv_cache_02_gb300 import HsError, RopeTable, tree_mask
from test_gpu_spec import DEV, check_append, check_tree, gqa, make_cache, mla, randn, random_tree


@pytest.mark.parametrize("dims", [(3,), (500,), (100, 300)])
def test_a_pairs_hand_overs_many_times(dims):
    """Shared latents, several portions and tiles a pair of CTAs, a node with infinite values in the dims of one CTA, of the
    other or of both: rows that do not see it have the bits of a clean cache in every one of many calls."""
    R, T, n = 6, 9, 4000
    cfg = mla(R)
    kv = make_cache(cfg, n + T, 16, seed=1)
    lens = [n - 613 * r for r in range(R)]
    mask = tree_mask(torch.tensor([[-1] + [max(-1, j - 2) for j in range(1, T)]] * R))  # even nodes and odd nodes
    only = {(r, i, h) for r in range(R) for i in (0, T - 1) for h in (0, 37)}
    q, clean = check_tree(cfg, kv, lens, T, mask, only=only)
    flat, table = kv.pages.view(-1, cfg.record_elems), kv.table.cpu()
    for r in range(R):
        for d in dims:
            flat[ref.row_of(table, r, lens[r] + 4, kv.pages.shape[1], 0), d] = float("inf")
    lt, m = torch.tensor(lens, dtype=torch.int64, device=DEV), mask.to(DEV)
    sees = torch.tensor([(mask[0, i, 0].item() >> 4) & 1 for i in range(T)], dtype=torch.bool)
    outs = [kv.tree_attn(q, lt, m) for _ in range(40)]
    assert kv.errors() == 0
    for out in outs:
        assert torch.equal(out[:, ~sees], clean[:, ~sees])
        assert torch.equal(out.view(torch.int16), outs[0].view(torch.int16))


# what a node sees is bad in a value, in a key (its score is NaN), or in both so that its score is -infinity; a latent's value
# is its key
@pytest.mark.parametrize("cfg,kind", [pytest.param(c, kind, id=f"{name}-{kind}") for name, c in [
    ("gqa", gqa(1)), ("gqa64", gqa(1, 8, 2, 64)), ("any", gqa(1, 4, 2, 80)), ("mla", mla(1)), ("any-latent", mla(1, 3, 128, 64))]
    for kind in ["value-inf", "value-nan", "key-nan", "minus-infinity"] if c.layout == 1 or not kind.startswith("value")])
@pytest.mark.parametrize("n", [60, 200, 600, 20000])
@pytest.mark.parametrize("node", [False, True])
def test_a_bad_entry_of_next_to_no_weight_is_seen(kind, cfg, n, node):
    """One entry's weight is all there is in 32 bits (the others are below 2^-150 of it); a bad entry that has none makes
    its dims, or with a NaN score its rows, infinite or NaN all the same, whether one worker holds the context or many."""
    T, lat = 3, cfg.layout == 0
    kv = make_cache(cfg, n + T, 16, seed=n)
    flat, table, page = kv.pages.view(-1, cfg.record_elems), kv.table.cpu(), kv.pages.shape[1]
    flat *= 0.125
    D, Hkv, dim, col = cfg.head_dim_qk, cfg.num_kv_heads, 9, 9 if lat else 3
    q = randn((1, T, cfg.num_q_heads, D), 5)
    q[..., 0], q[..., col] = 8.0, -1.0
    row = lambda p: ref.row_of(table, 0, p, page, 0)  # noqa: E731
    for g in range(Hkv):  # scores of 8 * 512 / sqrt(D), 170 and more, against a few: 2^-245 at the most
        flat[row(n - 3), g * (D + cfg.head_dim_v)] = 512.0
    at = n + 1 if node else 7
    key = 0 if lat else (Hkv - 1) * (D + cfg.head_dim_v)  # of the last KV head
    where = {"value-inf": [(key + D + dim, "inf")], "value-nan": [(key + D + dim, "nan")], "key-nan": [(key + col, "nan")],
             "minus-infinity": [(key + col, "inf")] + ([] if lat else [(key + D + dim, "inf")])}[kind]
    for e, _ in where:
        flat[row(at), e] = 0.0
    parents = torch.tensor([[-1, 0, 1]])
    lens, mask = torch.tensor([n], dtype=torch.int64, device=DEV), tree_mask(parents)
    _, clean = check_tree(cfg, kv, [n], T, mask, q=q)
    for e, x in where:
        flat[row(at), e] = float(x)
    out = kv.tree_attn(q, lens, mask.to(DEV))
    assert kv.errors() == 0
    sees = torch.tensor([not node or i >= 1 for i in range(T)])
    heads = torch.arange(cfg.num_q_heads) // (cfg.num_q_heads // Hkv) == Hkv - 1
    assert torch.equal(out[0, ~sees], clean[0, ~sees]) and torch.equal(out[0, :, ~heads], clean[0, :, ~heads])
    hit = out[0, sees][:, heads]
    if kind == "key-nan":
        assert bool(hit.isnan().all())
        return
    assert not bool(torch.isfinite(hit[..., dim]).any())
    # the other dims: as without the entry, whose weight is nothing (its score was a few, it is that or -infinity)
    hit, same = hit.clone(), clean[0, sees][:, heads].clone()
    hit[..., dim] = same[..., dim] = 0
    assert torch.equal(hit, same)


@pytest.mark.parametrize("dim", [5, 300, 511, 570])
def test_one_bad_value_of_a_latent_reaches_every_row_that_sees_it(dim):
    """A NaN in a node's latent makes every (node, head) that sees it NaN.  Minus infinity does where the query is
    negative there (the score is infinity); where it is positive the score is -infinity: the row is as without the node,
    but for the dim itself when it is one of the value's."""
    T, n, sick = 11, 150, 4
    cfg = mla(1)
    kv = make_cache(cfg, n + T, 16, seed=dim)
    mask = tree_mask(torch.tensor([[-1] + [max(-1, j - 2) for j in range(1, T)]]))
    q, clean = check_tree(cfg, kv, [n], T, mask, seed=dim)
    without = mask.clone()
    without[0, :, 0] &= ~(1 << sick)
    flat, table = kv.pages.view(-1, cfg.record_elems), kv.table.cpu()
    rows = [ref.row_of(table, 0, p, kv.pages.shape[1], 0) for p in range(n + T)]
    want, bound = ref.tree(cfg, [flat[rows[:n]]], [flat[rows[n:]]], q, without.tolist(), [T], cfg.default_scale)
    lens = torch.tensor([n], dtype=torch.int64, device=DEV)
    sees = torch.tensor([(mask[0, i, 0].item() >> sick) & 1 for i in range(T)], dtype=torch.bool, device=DEV)
    at = (rows[n + sick], dim)
    flat[at] = float("nan")
    out = kv.tree_attn(q, lens, mask.to(DEV))
    assert torch.equal(out[0, ~sees], clean[0, ~sees]) and bool(out[0, sees].isnan().all())
    flat[at] = -float("inf")
    out = kv.tree_attn(q, lens, mask.to(DEV))
    assert torch.equal(out[0, ~sees], clean[0, ~sees])
    up = q[0, :, :, dim] < 0  # [T][heads]
    assert bool((q[0, :, :, dim] != 0).all())
    assert bool(out[0][sees[:, None] & up].isnan().all())
    down = sees[:, None] & ~up
    got, w, b = out[0][down].double(), want[0][down], bound[0][down]
    keep = torch.arange(cfg.head_dim_v, device=DEV) != dim
    assert bool(((got - w).abs() <= b)[:, keep].all()) and (dim >= 512 or not bool(torch.isfinite(got[:, dim]).any()))


# tokens a CTA: 2 below 456 * 4 tokens, else 4; the last CTA of each with fewer
@pytest.mark.parametrize("N", [1031, 1825, 1827, 8191])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("cfg,rd,q_dim", [(gqa(2, 6, 2, 64), 32, 64), (gqa(2), 16, 128), (mla(2, 5), 64, 64)],
                         ids=["gqa64", "gqa", "latent"])
def test_append_of_several_tokens_a_cta(cfg, rd, q_dim, interleaved, N):
    inv = [10000.0 ** (-j / (rd // 2)) for j in range(rd // 2)]
    check_append(cfg, N, [N // 3, N - N // 3 - 5], [9, 4], 16, RopeTable(rd, interleaved=interleaved), inv, interleaved,
                 q_dim=q_dim, lead=2)


@pytest.mark.parametrize("R", [33, 64, 1025])
@pytest.mark.parametrize("most", [1, 9])
def test_append_to_many_requests(R, most):
    """Requests are searched 32 places at a time: runs of requests without a token, before, between and behind the others
    and across those places, padding tokens before and behind."""
    counts = [0 if r < 3 or r >= R - 2 or (r // 5) % 3 == 1 or 28 < r % 32 < 31 else 1 + r % most for r in range(R)]
    inv = [1.0, 0.5, 0.25, 0.1, 1e-2, 1e-3, 1e-4, 1e-5]
    check_append(gqa(R, 2, 1, 24), sum(counts) + 7, counts, [r % 11 for r in range(R)], 5, RopeTable(16, inv_freq=inv), inv, False,
                 q_dim=16, off=8, lead=4)


def test_an_output_over_the_queries_is_refused():
    cfg, T = gqa(2), 4
    kv = make_cache(cfg, 60, 16, seed=1)
    both = randn((4, T, cfg.num_q_heads, cfg.head_dim_qk), 2)
    q, lens, mask = both[:2], torch.tensor([50, 3], dtype=torch.int64, device=DEV), tree_mask(random_tree(2, T, 1)).to(DEV)
    for out in (q, both[1:3]):
        with pytest.raises(HsError):
            kv.tree_attn(q, lens, mask, out=out)
    assert torch.equal(kv.tree_attn(q, lens, mask, out=both[2:]), kv.tree_attn(q, lens, mask))  # right behind them
