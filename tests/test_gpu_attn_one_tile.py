"""Attention over rows, and parts of rows, of exactly one tile of 32 keys: one
CTA of the pair then owns no tile, and takes the other's P over a place where
its own Q has landed."""
import numpy as np
import pytest
import torch

from gpu_util import lib
from test_gpu_q8 import _attend, _cache, _check, _f64, _indices, _t

pytestmark = pytest.mark.gpu
DEV = "cuda"
REPEATS = 30


def _q(g, R, H):
    return torch.as_tensor(g.standard_normal((R, H, 576)).astype(np.float32)).to(torch.bfloat16)


def _attend_bf16(hs, q, kv, idx, scale):
    R, H, _ = q.shape
    out = torch.full((R, H, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((R, H), float("nan"), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    hs.hs_sparse_attn_decode(q, kv, idx, scale, out, lse=lse, status=st)
    assert int(st.item()) == 0
    return out, lse


@pytest.mark.parametrize("R,H,K", [(1, 128, 1), (2, 17, 32), (5, 128, 31), (90, 128, 32), (200, 130, 20), (400, 64, 7)])
@pytest.mark.parametrize("kind", ["q8", "bf16"])
def test_rows_of_one_tile(kind, R, H, K):
    hs = lib()
    g = np.random.default_rng(R * 1009 + H * 7 + K)
    rows, values = _cache(g, 500)
    idx = _indices(g, R, K, 500, 0.1)
    idx[0, 0] = 3
    q = _q(g, R, H)
    cache = _t(rows) if kind == "q8" else torch.as_tensor(values).to(torch.bfloat16).to(DEV)
    call = _attend if kind == "q8" else _attend_bf16
    dq, di = q.to(DEV), _t(idx)
    out, lse = call(hs, dq, cache, di, 1 / 24)
    _check(out, lse, _f64(q), values, idx, 1 / 24)
    for _ in range(REPEATS):
        again, lse2 = call(hs, dq, cache, di, 1 / 24)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("R,H,K", [(1, 128, 672), (1, 17, 670), (2, 128, 653), (1, 256, 1313)])
def test_a_last_part_of_one_tile(R, H, K):
    """21 tiles in parts of 5, 5, 5, 5 and 1 (42: 5 x 8, 2), with a workspace."""
    hs = lib()
    g = np.random.default_rng(R * 1013 + H * 7 + K)
    rows, values = _cache(g, 900)
    idx = _indices(g, R, K, 900, 0.05)
    q = _q(g, R, H)
    ws = torch.full((32 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    cache, dq, di = _t(rows), q.to(DEV), _t(idx)
    out, lse = _attend(hs, dq, cache, di, 1 / 24, ws)
    _check(out, lse, _f64(q), values, idx, 1 / 24)
    for _ in range(REPEATS):
        again, lse2 = _attend(hs, dq, cache, di, 1 / 24, ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
