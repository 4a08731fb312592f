"""The bounded waits of the attention over shared prefixes, exercised without any GPU fault: a test hook has a
barrier wait for an arrival that nothing makes, the waits run to their limit of about a second, and the call reports it and
leaves everything usable."""
import time

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import batch_ref as ref
from hierarchical_kv_cache_02_gb300 import DEVERR_TIMEOUT
from test_gpu_batch import DEV, gqa, mla
from test_gpu_prefix import check

CASES = [
    pytest.param(lambda R: gqa(R), 16, id="gqa-boxes"),
    pytest.param(lambda R: gqa(R), 7, id="gqa-records"),
    pytest.param(lambda R: gqa(R, 28, 4, 64), 32, id="gqa64-boxes"),
    pytest.param(lambda R: gqa(R, 128, 1), 16, id="gqa-two-row-tiles"),
    pytest.param(lambda R: mla(R), 16, id="latent-boxes"),
    pytest.param(lambda R: mla(R), 7, id="latent-records"),
    pytest.param(lambda R: mla(R, 24), 64, id="latent-few-rows"),
]


@pytest.mark.parametrize("shape,page", CASES)
@pytest.mark.parametrize("lists", [0, 1])
def test_a_prefix_attention_gives_up_reports_and_leaves_the_cache_usable(shape, page, lists):
    """Every worker misses an arrival of its first tile: their producers, products and softmax all have work in flight."""
    R = 5
    cfg = shape(R)
    groups, prefix, lens = [0, 3], [9000], [9000, 9300, 9100, 4000, 700]
    kv, q, out, acc = check(cfg, groups, prefix, lens, page, lists=lists, only={(0, 0), (2, 1), (4, 3)}, seed=3)
    gt, pt = torch.tensor(groups, dtype=torch.int32, device=DEV), torch.tensor(prefix, device=DEV)
    lt = torch.tensor(lens, device=DEV)
    pages = kv.pages.clone()
    w = torch.zeros_like(acc) if lists else None
    kv.debug_stall_next()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    kv.prefix_attn(q, lt, groups=gt, prefix=pt, weights=w)  # its output is undefined
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert kv.errors(reset=True) == DEVERR_TIMEOUT
    # the wait ran for its limit; clean-up waits for what is in flight, each with a limit of a second of its own
    assert 0.9 <= elapsed <= 5.0, elapsed
    # the hook was consumed, and the cache is as it was
    assert ref.same(kv.pages, pages)
    for _ in range(3):
        w = torch.rand(acc.shape, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV) if lists else None
        assert ref.same(kv.prefix_attn(q, lt, groups=gt, prefix=pt, weights=w), out)
    assert kv.errors() == 0


def test_the_hook_is_of_the_calling_thread_and_waits_for_the_tensor_cores():
    import threading

    kv, q, out, _ = check(gqa(3), [0], [], [60, 70, 200])
    lens = torch.tensor([60, 70, 200], dtype=torch.int64, device=DEV)
    t = threading.Thread(target=kv.debug_stall_next)
    t.start()
    t.join()
    assert ref.same(kv.prefix_attn(q, lens), out) and kv.errors() == 0
    kv.debug_stall_next()
    check(gqa(3, 4, 2, 80), [0], [], [60, 70, 200])  # on CUDA cores: nothing waits
    kv.prefix_attn(q, lens)
    assert kv.errors(reset=True) == DEVERR_TIMEOUT
    assert ref.same(kv.prefix_attn(q, lens), out) and kv.errors() == 0
