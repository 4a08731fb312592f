"""The entry points of a batch's decode step refuse bad arguments on the host, before anything touches a device."""
import ctypes

import pytest

pytest.importorskip("torch")

from hierarchical_kv_cache_02_gb300 import _lib, build
from test_spec_host import BAD_PAGES, BAD_SHAPES, OK_PTR, append, paged, shape


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return _lib.load()


def norm(**change):
    base = dict(d_k_weight=OK_PTR, k_weight_head_stride=0, d_q_weight=OK_PTR, q_weight_head_stride=128, k_weight_type=0, q_weight_type=1,
                eps=1e-6, axes=1, d_axis=None)
    base.update(change)
    return _lib.hs_norm_args(**base)


def evict(**change):
    base = dict(d_len=OK_PTR, d_weights=OK_PTR, d_weights_out=OK_PTR, d_len_out=OK_PTR, d_first=None, capacity=64, lists=8, keep=32, first=4,
                recent=8, d_workspace=OK_PTR, workspace_bytes=1 << 40)
    base.update(change)
    return _lib.hs_evict_args(**base)


def prefix(**change):
    base = dict(d_q=OK_PTR, d_len=OK_PTR, d_groups=OK_PTR, d_prefix=OK_PTR, groups=2, scale=0.1, d_weights=OK_PTR, capacity=64, lists=8, decay=1.0,
                d_out=OK_PTR << 8, d_workspace=OK_PTR, workspace_bytes=1 << 40)
    base.update(change)
    return _lib.hs_prefix_args(**base)


def ref(x):
    return ctypes.byref(x)


@pytest.mark.parametrize("change", BAD_SHAPES)
def test_bad_shapes(lib, change):
    c, kv = shape(**change), paged()
    assert lib.hs_append_normed(ref(c), ref(kv), ref(append()), ref(norm()), None) == _lib.HS_ERR_CONFIG
    assert lib.hs_evict(ref(c), ref(kv), ref(evict()), None) == _lib.HS_ERR_CONFIG
    assert lib.hs_evict_workspace(ref(c), 1, 8) == _lib.HS_ERR_CONFIG
    assert lib.hs_prefix_attn(ref(c), ref(kv), ref(prefix()), None) == _lib.HS_ERR_CONFIG
    assert lib.hs_prefix_attn_workspace(ref(c), ref(kv), 1, 0) == _lib.HS_ERR_CONFIG


@pytest.mark.parametrize("change", BAD_PAGES)
def test_bad_pages(lib, change):
    c, kv = shape(), paged(**change)
    assert lib.hs_append_normed(ref(c), ref(kv), ref(append()), ref(norm()), None) == _lib.HS_ERR_ARG
    assert lib.hs_evict(ref(c), ref(kv), ref(evict()), None) == _lib.HS_ERR_ARG
    assert lib.hs_prefix_attn(ref(c), ref(kv), ref(prefix()), None) == _lib.HS_ERR_ARG
    assert lib.hs_prefix_attn_workspace(ref(c), ref(kv), 1, 0) == _lib.HS_ERR_ARG


@pytest.mark.parametrize("change", [
    dict(d_q=None), dict(d_q=OK_PTR + 8), dict(d_len=None), dict(d_len=OK_PTR + 4), dict(d_groups=None), dict(d_groups=OK_PTR + 2),
    dict(d_prefix=None), dict(d_prefix=OK_PTR + 4), dict(groups=-1), dict(groups=3), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(scale=2.5e38), dict(d_weights=OK_PTR + 2), dict(capacity=0), dict(capacity=1 << 31), dict(lists=2), dict(lists=0),
    dict(decay=float("nan")), dict(decay=float("inf")), dict(d_out=None), dict(d_out=(OK_PTR << 8) + 8), dict(d_out=OK_PTR + 64),
    dict(d_workspace=OK_PTR + 8)])
def test_bad_prefixes(lib, change):
    assert lib.hs_prefix_attn(ref(shape()), ref(paged()), ref(prefix(**change)), None) == _lib.HS_ERR_ARG


def test_bad_workspaces_of_prefixes(lib):
    c, kv = shape(), paged()
    for groups in (-1, 3):
        assert lib.hs_prefix_attn_workspace(ref(c), ref(kv), groups, 0) == _lib.HS_ERR_ARG
    assert lib.hs_prefix_attn_workspace(ref(c), None, 0, 0) == _lib.HS_ERR_ARG
    assert lib.hs_prefix_attn_workspace(None, ref(kv), 0, 0) == _lib.HS_ERR_ARG


@pytest.mark.parametrize("change", [
    dict(d_k_weight=OK_PTR + 4), dict(d_q_weight=OK_PTR + 8), dict(k_weight_head_stride=-128), dict(q_weight_head_stride=4),
    dict(k_weight_type=2), dict(q_weight_type=-1), dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(axes=0), dict(axes=5), dict(axes=2)])
def test_bad_norms(lib, change):
    assert lib.hs_append_normed(ref(shape()), ref(paged()), ref(append()), ref(norm(**change)), None) == _lib.HS_ERR_ARG


@pytest.mark.parametrize("change", [dict(d_q=None), dict(q_dim=64), dict(d_k=None), dict(d_cu=None), dict(num_tokens=-1)])
def test_bad_appends_with_norms(lib, change):
    assert lib.hs_append_normed(ref(shape()), ref(paged()), ref(append(**change)), ref(norm()), None) == _lib.HS_ERR_ARG


def test_axes_need_positions_and_latents_have_no_norm_of_queries(lib):
    args = append(d_rope_pos=None)
    assert lib.hs_append_normed(ref(shape()), ref(paged()), ref(args), ref(norm(axes=2, d_axis=OK_PTR)), None) == _lib.HS_ERR_ARG
    c = shape(layout=0, num_kv_heads=1, num_q_heads=64, head_dim_qk=576, head_dim_v=512)
    args = append(d_v=None, q_dim=576, q_head_stride=576, q_token_stride=36864, q_out_head_stride=576, q_out_token_stride=36864)
    assert lib.hs_append_normed(ref(c), ref(paged()), ref(args), ref(norm()), None) == _lib.HS_ERR_ARG


@pytest.mark.parametrize("change", [
    dict(d_len=None), dict(d_len=OK_PTR + 4), dict(d_weights=None), dict(d_weights=OK_PTR + 2), dict(d_weights_out=None),
    dict(d_len_out=None), dict(d_len_out=OK_PTR + 8), dict(d_first=OK_PTR + 4), dict(capacity=0), dict(capacity=1 << 31), dict(lists=2),
    dict(lists=0), dict(keep=0), dict(keep=-1), dict(recent=-1), dict(recent=33), dict(first=-1), dict(first=25), dict(keep=2**31 - 1),
    dict(d_weights_out=OK_PTR + 64), dict(d_weights=OK_PTR + 64), dict(d_workspace=OK_PTR + 8)])
def test_bad_evictions(lib, change):
    assert lib.hs_evict(ref(shape()), ref(paged()), ref(evict(**change)), None) == _lib.HS_ERR_ARG


def test_workspace_of_evictions(lib):
    need = lib.hs_evict_workspace(ref(shape()), 8, 32)
    assert need > 0
    for change in (dict(workspace_bytes=need - 1), dict(d_workspace=None)):
        assert lib.hs_evict(ref(shape()), ref(paged()), ref(evict(**change)), None) == _lib.HS_ERR_SCRATCH
    for lists, keep in ((2, 8), (1, 0), (1, 2**31 - 1)):
        assert lib.hs_evict_workspace(ref(shape()), lists, keep) == _lib.HS_ERR_ARG


def test_null_arguments(lib):
    c, kv = shape(), paged()
    assert lib.hs_append_normed(ref(c), ref(kv), None, ref(norm()), None) == _lib.HS_ERR_ARG
    assert lib.hs_append_normed(ref(c), ref(kv), ref(append()), None, None) == _lib.HS_ERR_ARG
    assert lib.hs_append_normed(None, ref(kv), ref(append()), ref(norm()), None) == _lib.HS_ERR_ARG
    assert lib.hs_evict(ref(c), None, ref(evict()), None) == _lib.HS_ERR_ARG
    assert lib.hs_evict(ref(c), ref(kv), None, None) == _lib.HS_ERR_ARG
    assert lib.hs_prefix_attn(ref(c), None, ref(prefix()), None) == _lib.HS_ERR_ARG
    assert lib.hs_prefix_attn(ref(c), ref(kv), None, None) == _lib.HS_ERR_ARG
