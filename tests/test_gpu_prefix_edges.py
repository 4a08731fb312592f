"""Attention over shared prefixes on the GPU: softmax warps that are a portion's end apart, and rows with more partials than
the join looks at in one round."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import batch_ref as ref
from test_gpu_batch import DEV, gqa, mla
from test_gpu_prefix import check


# a latent's CTA of 64 rows: 32 rows or fewer have two of its four softmax warps without one, which run ahead at a portion's end
@pytest.mark.parametrize("heads", [17, 24, 32, 40, 88, 96, 152])
@pytest.mark.parametrize("weigh", [False, True])
def test_latent_portions_with_few_rows(heads, weigh):
    """Many short portions a worker; a sample of the rows is compared, and all of them with those of equal calls."""
    R, most = 400, 200
    cfg = mla(R, heads)
    g = torch.Generator().manual_seed(heads)
    lens = [1 + int(x) for x in torch.randint(0, most, (R,), generator=g)]
    lens[0] = most
    only = {(a % R, b % heads) for a, b in torch.randint(0, 10**9, (200, 2), generator=g).tolist()}
    kv, q, out, acc = check(cfg, [0], [], lens, 16, lists=1 if weigh else 0, only=only, seed=heads)
    lt = torch.tensor(lens, device=DEV)
    for _ in range(20):
        w = torch.zeros_like(acc) if weigh else None
        assert ref.same(kv.prefix_attn(q, lt, weights=w), out)
        if weigh:
            # A row's weights add up to 1, as powers and sum are of the same scores: a score of magnitude s is rounded once
            # more for the weights, and less the maximum (2 s 2^-24, s < 300 here), powers are off by 2^-22 on both sides,
            # sums of 200 terms by 200 2^-24, quotient and product by 2^-23: less than 2^-14 in all, and as much for the reading.
            total = w.double().sum(dim=2)[:, 0]
            assert bool(((total - heads).abs() <= heads * 2.0**-13).all())
    assert kv.errors() == 0


# an item over nearly all workers leaves each of its rows a partial or two from each: over 64 of them
@pytest.mark.parametrize("cfg,groups,prefix,lens", [
    (mla(1), [0], [], [33000]),
    (mla(1, 5), [0, 1], [20000], [33000]),
    (mla(2), [0, 2], [30000], [36000, 30500]),
    (mla(2, 63), [0, 1], [12000], [36000, 12]),
    (gqa(1, 8, 1), [0], [], [40000]),
    (gqa(1, 128, 1, 64), [0], [], [40000]),
    (gqa(2, 8, 1), [0, 2], [40000], [52000, 41000]),
    (gqa(2, 7, 1, 64), [0, 2], [40001], [80000, 40001]),
    (gqa(3, 128, 1), [0, 3], [50000], [50100, 50000, 60000]),
], ids=["latent", "latent-5-heads", "latent-pair", "latent-63-heads", "gqa", "gqa64-128-heads", "gqa-pair", "gqa64-pair", "gqa-two-row-tiles"])
@pytest.mark.parametrize("weigh", [False, True])
def test_rows_of_many_partials(cfg, groups, prefix, lens, weigh):
    kv, q, out, _ = check(cfg, groups, prefix, lens, 64, lists=1 if weigh else 0, seed=len(lens))
    gt, pt = torch.tensor(groups, dtype=torch.int32, device=DEV), torch.tensor(prefix, dtype=torch.int64, device=DEV)
    lt = torch.tensor(lens, device=DEV)
    for _ in range(5):
        assert ref.same(kv.prefix_attn(q, lt, groups=gt, prefix=pt), out)  # with weights or without
