"""More refusals of the speculative-decoding entry points on the host, before anything touches a device."""
import ctypes

import pytest

from hierarchical_kv_cache_02_gb300 import _lib
from test_spec_host import append, lib, paged, shape, tree  # noqa: F401 (lib: a fixture)


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_a_scale_that_overflows_in_base_two(lib, scale):  # noqa: F811
    """Scores are taken times scale * log2(e): where that is infinite, a score of 0 would be NaN."""
    c, kv = shape(), paged()
    a = tree(scale=scale, d_out=1 << 40)
    assert lib.hs_tree_attn(ctypes.byref(c), ctypes.byref(kv), ctypes.byref(a), None) == _lib.HS_ERR_ARG


@pytest.mark.parametrize("off", [0, 16, -16, 2 * 2 * 4 * 32 * 128 - 16, -(2 * 2 * 4 * 32 * 128 - 16)])
def test_an_output_over_the_queries(lib, off):  # noqa: F811
    """Rows are written while other rows' queries are still read: in place is refused."""
    c, kv, q = shape(), paged(), 1 << 40
    assert lib.hs_tree_attn(ctypes.byref(c), ctypes.byref(kv), ctypes.byref(tree(d_q=q, d_out=q + off)), None) == _lib.HS_ERR_ARG


@pytest.mark.parametrize("change", [dict(q_out_token_stride=8192), dict(q_token_stride=8192), dict(q_head_stride=0),
                                    dict(q_out_token_stride=128, q_out_head_stride=512)])
def test_a_query_rotated_in_place_keeps_its_strides(lib, change):  # noqa: F811
    """d_q_out may be d_q: then with the same strides, or a query would be overwritten before it is read."""
    c, kv = shape(), paged()
    assert lib.hs_append_rotated(ctypes.byref(c), ctypes.byref(kv), ctypes.byref(append(**change)), None) == _lib.HS_ERR_ARG
