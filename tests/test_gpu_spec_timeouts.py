"""The tree attentions' bounded waits, exercised without any GPU fault: a test hook leaves one barrier arrival out, the
waits for it run to their limit of about a second, and the call reports it and leaves everything usable."""
import time

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from hierarchical_kv_cache_02_gb300 import DEVERR_TIMEOUT, LAYOUT_GQA, LAYOUT_MLA, HsConfig, HsError, HsPool, inputs, tree_mask
from hierarchical_kv_cache_02_gb300._lib import STALL_TREE

DEV = "cuda:0"


# one row tile (two workers a CTA), two row tiles (one), pairs of CTAs
@pytest.mark.parametrize("layout,T", [(LAYOUT_GQA, 8), (LAYOUT_GQA, 64), (LAYOUT_MLA, 5)], ids=["gqa", "gqa-wide", "latent"])
def test_a_tree_attention_gives_up_reports_and_leaves_the_pool_usable(layout, T):
    R, ctx, k = 3, 3000, 2048
    shape = dict(num_q_heads=32, num_kv_heads=8, head_dim_qk=128, head_dim_v=128)
    if layout == LAYOUT_MLA:
        shape = dict(num_q_heads=64, num_kv_heads=1, head_dim_qk=576, head_dim_v=512)
    cfg = HsConfig(num_requests=R, num_layers=1, capacity=ctx, layout=layout, top_k=k, buffer_slots=k, **shape)
    pool = HsPool(cfg)
    hist = inputs.normal_bf16((R, ctx, cfg.record_elems), seed=1)
    for r in range(R):
        pool.prefill(r, 0, 0, hist[r])
    g = torch.Generator().manual_seed(2)
    locs = pool.resolve(0, torch.stack([torch.randperm(ctx, generator=g)[:k] for _ in range(R)]).to(torch.int32).to(DEV))
    q = inputs.normal_bf16((R, T, cfg.num_q_heads, cfg.head_dim_qk), seed=3).to(DEV)
    drafts = inputs.normal_bf16((R, T, cfg.record_elems), seed=4).to(DEV)
    mask = tree_mask(torch.arange(T).repeat(R, 1) - 1).to(DEV)
    first = pool.tree_attn(0, q, locs, drafts, mask)
    torch.cuda.synchronize()
    assert pool.stats()["error_bits"] == 0
    pool.debug_stall_next(STALL_TREE)
    t0 = time.perf_counter()
    pool.tree_attn(0, q, locs, drafts, mask)  # its output is undefined
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert pool.stats(reset=True)["error_bits"] == DEVERR_TIMEOUT
    # the wait ran for its limit; clean-up waits for what is in flight, each with a limit of a second of its own
    assert 0.9 <= elapsed <= 5.0, elapsed
    # the hook was consumed, and the pool's buffers are as they were
    assert torch.equal(pool.tree_attn(0, q, locs, drafts, mask), first)
    assert pool.stats()["error_bits"] == 0
    with pytest.raises(HsError):
        pool.debug_stall_next(16)
    pool.close()
