"""Attention over q8 rows behind the calls that write what it reads, with no
wait of the host between them: indices from hs_resolve_topk (which lets the
attention start beside it), rows from hs_quant_rows, parts from the call's own
first kernel. Every call must see its own step's values, in places that held an
earlier step's."""
import numpy as np
import pytest
import torch

from oracle import hs_oracle as O
from gpu_util import lib
from test_gpu_q8 import _check, _f64, _t

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("H", [128, 20, 16])
def test_every_step_sees_its_own_values(H, split):
    hs = lib()
    g = np.random.default_rng(19 + H)
    B, L, bs, K, steps = 4, 900, 64, 300, 8
    nblk = (L + bs) // bs + 1
    n = B * nblk * bs
    bt = g.permutation(B * nblk).reshape(B, nblk).astype(np.int32)
    clen = np.full(B, L, np.int32)
    req = np.arange(B, dtype=np.int32)
    d_req, d_clen, d_bt = _t(req), _t(clen), _t(bt)
    rows = [g.standard_normal((n, 576)).astype(np.float32) for _ in range(steps)]
    topks = [np.stack([g.permutation(L)[:K] for _ in range(B)]).astype(np.int32) for _ in range(steps)]
    qs = [torch.as_tensor(g.standard_normal((B, H, 576)).astype(np.float32)).to(torch.bfloat16) for _ in range(steps)]
    d_rows, d_topks, d_qs = [_t(r) for r in rows], [_t(t) for t in topks], [q.to(DEV) for q in qs]
    cache = torch.zeros((n, 656), dtype=torch.uint8, device=DEV)
    topk = torch.zeros((B, K), dtype=torch.int32, device=DEV)
    idx = torch.zeros_like(topk)
    ws = torch.full((32 << 20,), 0xFF, dtype=torch.uint8, device=DEV) if split else None
    outs = [torch.empty((B, H, 512), dtype=torch.bfloat16, device=DEV) for _ in range(steps)]
    lses = [torch.empty((B, H), device=DEV) for _ in range(steps)]
    twice = [torch.empty_like(o) for o in outs]
    torch.cuda.synchronize()
    for s in range(steps):
        topk.copy_(d_topks[s])
        hs.hs_quant_rows(d_rows[s], cache)
        hs.hs_resolve_topk(d_req, d_clen, d_bt, topk, bs, bs, idx)
        hs.hs_sparse_attn_decode_q8(d_qs[s], cache, idx, 1 / 24, outs[s], lse=lses[s], workspace=ws)
        # the rows written last: by the kernel right before the attention
        hs.hs_quant_rows(d_rows[(s + 1) % steps], cache)
        hs.hs_quant_rows(d_rows[s], cache)
        hs.hs_sparse_attn_decode_q8(d_qs[s], cache, idx, 1 / 24, twice[s], workspace=ws)
    torch.cuda.synchronize()
    for s in range(steps):
        e_idx, _, _ = O.resolve_topk(req, clen, bt, topks[s], bs, bs)
        values = O.q8_values(O.q8_quantise(rows[s].astype(np.float64)))
        _check(outs[s], lses[s], _f64(qs[s]), values, e_idx, 1 / 24)
        assert torch.equal(outs[s], twice[s])
