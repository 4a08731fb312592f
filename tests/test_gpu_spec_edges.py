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
