"""Edges of the speculative-decoding operators on the GPU that the operators' own tests leave out."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import spec_ref as ref
from hierarchical_kv_cache_02_gb300 import tree_mask
from test_gpu_spec import DEV, check_tree, gqa, make_cache, mla, randn, random_tree


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


# what a node sees is bad in a value, in a key (its score is NaN), or in both so that its score is -infinity
@pytest.mark.parametrize("kind", ["value-inf", "value-nan", "key-nan", "minus-infinity"])
@pytest.mark.parametrize("cfg", [gqa(1), gqa(1, 8, 2, 64), gqa(1, 4, 2, 80), mla(1), mla(1, 3, 128, 64)],
                         ids=["gqa", "gqa64", "any", "mla", "any-latent"])
@pytest.mark.parametrize("n", [60, 200, 600, 20000])
@pytest.mark.parametrize("node", [False, True])
def test_a_bad_entry_of_next_to_no_weight_is_seen(kind, cfg, n, node):
    """One entry's weight is all there is in 32 bits (the others are below 2^-150 of it); a bad entry that has none makes
    its dims, or with a NaN score its rows, infinite or NaN all the same, whether one worker holds the context or many."""
    T, lat = 3, cfg.layout == 0
    if lat and kind.startswith("value"):
        pytest.skip("a latent's value is its key")
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
