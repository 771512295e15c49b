"""Scales at the ends of their range: 0 (and what is smaller than the smallest normal
number) weighs all selected keys alike, masked ones not at all; negative and infinite
ones are refused before a swap-in has begun."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_util import lib
from test_gpu_q4 import _check, _f64, _indices, _q, _t

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45, 1e-39])
@pytest.mark.parametrize("R,H,K,pad", [(3, 128, 300, 0.3), (2, 16, 33, 0.0), (2, 130, 64, 0.0), (2, 20, 5, 0.9)])
def test_scale_zero_is_the_mean(R, H, K, pad, scale):
    hs = lib()
    g = np.random.default_rng(R * 101 + H + K)
    kv = torch.as_tensor(g.standard_normal((400, 576)).astype(np.float32)).to(torch.bfloat16)
    idx = _indices(g, R, K, 400, pad)
    idx[0] = -1
    q = _q(g, R, H)
    dq, dkv, di = q.to(DEV), kv.to(DEV), _t(idx)
    flags = torch.ones(R, dtype=torch.int32, device=DEV)
    calls = (lambda o, l: hs.hs_sparse_attn_decode(dq, dkv, di, scale, o, lse=l),
             lambda o, l: hs.hs_sparse_attn_decode_mixed(dq, dkv, dkv[:1], None, flags, di, scale, o, lse=l))
    for call in calls:
        out = torch.full((R, H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((R, H), 7.0, device=DEV)
        call(out, lse)
        _check(out, lse, _f64(q), _f64(kv), idx, 0.0)


def test_refused_scales_leave_a_step_undone():
    hs = lib()
    B, S, n_step, bs, max_ctx = 2, 8, 2, 4, 32
    hbt = np.arange(B * 8, dtype=np.int32).reshape(B, 8)
    pool = W.host_pool_tensor(B * 32, 5, device=DEV)
    hot = torch.zeros((B * (S + n_step), 576), dtype=torch.bfloat16, device=DEV)
    buf = hs.HsBuffer(B, S, n_step, max_ctx, bs, hot, pool, _t(hbt))
    req, clen = _t(np.array([0, 1], np.int32)), _t(np.array([21, 22], np.int32))
    kv_len = _t(np.array([20, 20], np.int32))
    topk = _t(np.array([[1, 2, -1]] * 2, np.int32))
    q = _q(np.random.default_rng(1), 2, 16).to(DEV)
    idx = torch.full((2, 3), -7, dtype=torch.int32, device=DEV)
    out = torch.full((2, 16, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    clock = buf.clock
    for bad in (-0.1, float("inf"), float("nan"), 3e38):
        with pytest.raises(hs.HisparseError):
            hs.hs_swap_in_attn_decode(buf, req, clen, kv_len, topk, q, bad, idx, out)
    torch.cuda.synchronize()
    assert buf.clock == clock and (idx == -7).all() and (out == 7).all()
    lse = torch.empty((2, 16), device=DEV)
    hs.hs_swap_in_attn_decode(buf, req, clen, kv_len, topk, q, 0.0, idx, out, lse=lse)
    torch.cuda.synchronize()
    at = idx.cpu().numpy()
    assert buf.clock == clock + 1 and hs.hs_get_status(buf) == 0 and (at[:, 2] == -1).all()
    _check(out, lse, _f64(q), _f64(hot), at, 0.0)
    buf.close()
