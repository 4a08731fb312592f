"""The speculative-decoding entry points refuse bad arguments on the host, before anything touches a device;
rotation tables and tree masks against their definitions."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

from hierarchical_kv_cache_02_gb300 import _lib, build
from hierarchical_kv_cache_02_gb300.pool import HsConfig

torch = pytest.importorskip("torch")

PI = Fraction("3.141592653589793238462643383279502884197169399375105820974944592307816406286208998628034825342117067982148086513282306647")
OK_PTR = 0x10000  # never read: the calls below are refused first


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return _lib.load()


def shape(**change):
    base = dict(num_requests=2, num_layers=1, capacity=10, top_k=8, buffer_slots=16)
    base.update(change)
    return HsConfig(**base).to_c()


def paged(**change):
    base = dict(d_pages=OK_PTR, d_table=OK_PTR, num_pages=8, page_tokens=16, max_pages=4, d_err=OK_PTR, cuda_device=0)
    base.update(change)
    return _lib.hs_paged_kv(**base)


def append(**change):
    base = dict(num_tokens=4, d_cu=OK_PTR, d_start=OK_PTR, d_rope_pos=OK_PTR, d_k=OK_PTR, k_token_stride=1024, k_head_stride=128,
                d_v=OK_PTR, v_token_stride=1024, v_head_stride=128, d_turns=OK_PTR, rotary_dim=64, rotary_offset=0,
                interleaved=0, d_q=OK_PTR, q_token_stride=4096, q_head_stride=128, d_q_out=OK_PTR, q_out_token_stride=4096,
                q_out_head_stride=128, q_dim=128)
    base.update(change)
    return _lib.hs_append_args(**base)


def tree(**change):
    base = dict(d_q=OK_PTR, d_len=OK_PTR, d_locs=None, top_k=0, d_mask=OK_PTR, d_nodes=None, nodes=4, scale=0.1, d_out=OK_PTR,
                d_workspace=OK_PTR, workspace_bytes=1 << 40)
    base.update(change)
    return _lib.hs_tree_args(**base)


BAD_SHAPES = [dict(num_requests=0), dict(num_requests=65536), dict(layout=2), dict(num_q_heads=30), dict(num_kv_heads=0),
              dict(num_q_heads=2048, num_kv_heads=1), dict(head_dim_qk=100), dict(head_dim_qk=0), dict(head_dim_v=584),
              dict(layout=0, num_kv_heads=2), dict(layout=0, num_kv_heads=1, head_dim_qk=64, head_dim_v=128)]
BAD_PAGES = [dict(d_pages=None), dict(d_pages=OK_PTR + 8), dict(d_table=OK_PTR + 2), dict(d_err=OK_PTR + 1), dict(num_pages=0),
             dict(page_tokens=0), dict(max_pages=0), dict(cuda_device=-1), dict(num_pages=1 << 28, page_tokens=16),
             dict(d_table=None, max_pages=5)]


@pytest.mark.parametrize("change", BAD_SHAPES)
def test_bad_shapes(lib, change):
    c, kv = shape(**change), paged()
    assert lib.hs_append_rotated(ctypes.byref(c), ctypes.byref(kv), ctypes.byref(append()), None) == _lib.HS_ERR_CONFIG
    assert lib.hs_tree_attn(ctypes.byref(c), ctypes.byref(kv), ctypes.byref(tree()), None) == _lib.HS_ERR_CONFIG
    assert lib.hs_keep_path(ctypes.byref(c), ctypes.byref(kv), OK_PTR, OK_PTR, 3, OK_PTR, None) == _lib.HS_ERR_CONFIG
    assert lib.hs_tree_attn_workspace(ctypes.byref(c), 4, 0) == _lib.HS_ERR_CONFIG


@pytest.mark.parametrize("change", BAD_PAGES)
def test_bad_pages(lib, change):
    c, kv = shape(), paged(**change)
    assert lib.hs_append_rotated(ctypes.byref(c), ctypes.byref(kv), ctypes.byref(append()), None) == _lib.HS_ERR_ARG
    assert lib.hs_tree_attn(ctypes.byref(c), ctypes.byref(kv), ctypes.byref(tree()), None) == _lib.HS_ERR_ARG
    assert lib.hs_keep_path(ctypes.byref(c), ctypes.byref(kv), OK_PTR, OK_PTR, 3, OK_PTR, None) == _lib.HS_ERR_ARG


@pytest.mark.parametrize("change", [
    dict(num_tokens=-1), dict(d_cu=None), dict(d_cu=OK_PTR + 1), dict(d_start=None), dict(d_start=OK_PTR + 4),
    dict(d_rope_pos=OK_PTR + 4), dict(d_k=None), dict(d_k=OK_PTR + 2), dict(k_token_stride=1020), dict(k_head_stride=-128),
    dict(d_v=None), dict(d_v=OK_PTR + 8), dict(v_token_stride=3), dict(v_head_stride=4), dict(rotary_dim=24),
    dict(rotary_dim=-16), dict(rotary_dim=144), dict(rotary_offset=72), dict(rotary_offset=4), dict(rotary_offset=-8),
    dict(interleaved=2), dict(d_turns=None), dict(d_turns=OK_PTR + 4), dict(d_q_out=None), dict(d_q=OK_PTR + 4),
    dict(d_q_out=OK_PTR + 2), dict(q_token_stride=7), dict(q_out_head_stride=12), dict(q_dim=96), dict(q_dim=0),
    dict(q_out_token_stride=0), dict(q_out_head_stride=0), dict(q_out_token_stride=128), dict(q_out_token_stride=4032),
    dict(q_out_token_stride=128, q_out_head_stride=384)])
def test_bad_appends(lib, change):
    c, kv = shape(), paged()
    assert lib.hs_append_rotated(ctypes.byref(c), ctypes.byref(kv), ctypes.byref(append(**change)), None) == _lib.HS_ERR_ARG


def test_a_shared_latent_has_no_values(lib):
    c = shape(layout=0, num_kv_heads=1, num_q_heads=64, head_dim_qk=576, head_dim_v=512)
    assert lib.hs_append_rotated(ctypes.byref(c), ctypes.byref(paged()), ctypes.byref(append()), None) == _lib.HS_ERR_ARG


@pytest.mark.parametrize("change", [
    dict(d_q=None), dict(d_q=OK_PTR + 8), dict(d_len=None), dict(d_len=OK_PTR + 4), dict(d_locs=OK_PTR, top_k=0),
    dict(d_locs=OK_PTR + 2, top_k=4), dict(d_mask=None), dict(d_mask=OK_PTR + 4), dict(d_nodes=OK_PTR + 1), dict(nodes=0),
    dict(nodes=257), dict(scale=float("nan")), dict(scale=float("inf")), dict(d_out=None), dict(d_out=OK_PTR + 4),
    dict(d_workspace=OK_PTR + 8)])
def test_bad_trees(lib, change):
    c, kv = shape(), paged()
    assert lib.hs_tree_attn(ctypes.byref(c), ctypes.byref(kv), ctypes.byref(tree(**change)), None) == _lib.HS_ERR_ARG


def test_null_arguments(lib):
    c, kv = shape(), paged()
    assert lib.hs_tree_attn(None, ctypes.byref(kv), ctypes.byref(tree()), None) == _lib.HS_ERR_ARG
    assert lib.hs_tree_attn(ctypes.byref(c), None, ctypes.byref(tree()), None) == _lib.HS_ERR_ARG
    assert lib.hs_tree_attn(ctypes.byref(c), ctypes.byref(kv), None, None) == _lib.HS_ERR_ARG
    assert lib.hs_append_rotated(ctypes.byref(c), ctypes.byref(kv), None, None) == _lib.HS_ERR_ARG
    assert lib.hs_pool_tree_attn(None, 0, ctypes.byref(tree()), OK_PTR, None) == _lib.HS_ERR_ARG
    for a in [(None, OK_PTR, 2, OK_PTR), (OK_PTR, None, 2, OK_PTR), (OK_PTR, OK_PTR, 2, None), (OK_PTR, OK_PTR, -1, OK_PTR),
              (OK_PTR, OK_PTR, 257, OK_PTR), (OK_PTR + 4, OK_PTR, 2, OK_PTR), (OK_PTR, OK_PTR + 2, 2, OK_PTR)]:
        assert lib.hs_keep_path(ctypes.byref(c), ctypes.byref(kv), *a, None) == _lib.HS_ERR_ARG
    assert lib.hs_tree_attn_workspace(None, 4, 0) == _lib.HS_ERR_ARG
    assert lib.hs_tree_attn_workspace(ctypes.byref(c), 0, 0) == _lib.HS_ERR_ARG
    assert lib.hs_tree_attn_workspace(ctypes.byref(c), 257, 0) == _lib.HS_ERR_ARG
    assert lib.hs_rope_turns(None, 3, None) == _lib.HS_ERR_ARG
    assert lib.hs_rope_turns(OK_PTR, -1, OK_PTR) == _lib.HS_ERR_ARG
    assert lib.hs_rope_turns(None, 0, None) == _lib.HS_OK


def test_turns_are_the_frequencies_over_a_whole_turn(lib):
    """Correctly rounded: half a step of 2^-64 of a turn (plus what 256 bits of 1 / (2 pi) leave: nothing to see)."""
    f = np.array([1.0, 0.5, 10000.0 ** (-1 / 64), 1e-9, 0.0, 3.0, 7.0, 1000.0, -0.25, -1e-30, 5e-324, 2.0**-64, 6.283185307179586,
                  2.0**32 - 1, 1e-15, 1e-25, -3.3e9], dtype=np.float64)
    t = np.empty(len(f), dtype=np.uint64)
    assert lib.hs_rope_turns(f.ctypes.data, len(f), t.ctypes.data) == _lib.HS_OK
    for x, got in zip(f.tolist(), t.tolist()):
        off = Fraction(got, 2**64) - Fraction(x) / (2 * PI)
        off -= round(off)  # a turn more or less is the same angle
        assert abs(off) <= Fraction(1, 2**65) + Fraction(1, 2**150), x
    for bad in (float("nan"), float("inf"), -float("inf"), 2.0**32):
        f[2] = bad
        assert lib.hs_rope_turns(f.ctypes.data, len(f), t.ctypes.data) == _lib.HS_ERR_ARG


@pytest.mark.parametrize("T", [1, 2, 5, 63, 64, 65, 130])
def test_tree_mask(T):
    from hierarchical_kv_cache_02_gb300 import tree_mask

    g = torch.Generator().manual_seed(T)
    parents = torch.stack([torch.arange(T) - 1] + [torch.tensor([-1] + [int(torch.randint(-1, j, (1,), generator=g))
                                                                        for j in range(1, T)]) for _ in range(2)])
    mask = tree_mask(parents)
    assert mask.shape == (3, T, (T + 63) // 64) and mask.dtype == torch.int64
    for r in range(3):
        for i in range(T):
            seen, j = set(), i
            while j >= 0:
                seen.add(j)
                j = int(parents[r, j])
            bits = {j for j in range(64 * mask.shape[2]) if (int(mask[r, i, j // 64]) >> (j % 64)) & 1}
            assert bits == seen
    with pytest.raises(ValueError):
        tree_mask(parents[0])
