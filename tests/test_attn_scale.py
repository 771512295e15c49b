"""Scales that no attention call can give a softmax for are refused on the host, before
anything touches a device."""
import ctypes

import pytest

import __graft_entry__ as G


@pytest.mark.parametrize("scale", [-1.0, -1e-30, float("nan"), float("inf"), -float("inf"), 2.0 ** 127 * 1.5])
def test_refused_scales(scale):
    G.build()
    import hisparse_top_sparse_gb300 as hs
    L = hs.lib()
    p, s = ctypes.c_void_p(1 << 20), ctypes.c_float(scale)
    assert L.hs_sparse_attn_decode(p, p, 10, p, 1, 16, 4, s, p, None, None, None) == hs.HS_ERR_INVALID_ARG
    assert b"scale" in L.hs_last_error_string()
    assert L.hs_sparse_attn_decode_mixed(p, p, 10, p, 10, None, p, 1, p, 1, 16, 4, s, p, None, None,
                                         None) == hs.HS_ERR_INVALID_ARG
    assert b"scale" in L.hs_last_error_string()
    for call in (L.hs_sparse_attn_decode_q8, L.hs_sparse_attn_decode_q4):
        assert call(p, p, 10, p, 1, 16, 4, s, p, None, None, 0, None, None) == hs.HS_ERR_INVALID_ARG
        assert b"scale" in L.hs_last_error_string()
