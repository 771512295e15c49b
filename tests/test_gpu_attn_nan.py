"""NaN in a selected row or in q: NaN in out and in lse, in every format, split and
kernel; heads and rows that it does not reach keep their bits."""
import numpy as np
import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
N, R = 300, 3
BAD = 250                      # the row that holds NaN


def _call(hs, kind, split, g):
    """The attention of a kind, over rows of which BAD holds a NaN."""
    x = torch.as_tensor(g.standard_normal((N, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    x[BAD, 37] = float("nan")
    if kind == "bf16":
        assert not split
        return lambda q, idx, out, lse: hs.hs_sparse_attn_decode(q, x, idx, 1 / 24, out, lse=lse)
    row, quant, attend = ((656, hs.hs_quant_rows, hs.hs_sparse_attn_decode_q8) if kind == "q8" else
                          (416, hs.hs_quant_rows_q4, hs.hs_sparse_attn_decode_q4))
    kv = torch.zeros((N, row), dtype=torch.uint8, device=DEV)
    quant(x, kv)
    ws = torch.full((32 << 20,), 0xFF, dtype=torch.uint8, device=DEV) if split else None
    return lambda q, idx, out, lse: attend(q, kv, idx, 1 / 24, out, lse=lse, workspace=ws)


CASES = [(kind, H, split) for kind in ("bf16", "q8", "q4") for H in (128, 20, 16, 5) for split in (False, True)
         if not (kind == "bf16" and split)]


@pytest.mark.parametrize("K", [1, 40, 1500])
@pytest.mark.parametrize("kind,H,split", CASES)
def test_nan_reaches_out_and_lse(kind, H, split, K):
    hs = lib()
    g = np.random.default_rng(H + K)
    call = _call(hs, kind, split, g)
    q = torch.as_tensor(g.standard_normal((R, H, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    clean = g.integers(0, BAD, size=(R, K)).astype(np.int32)
    clean[0, K // 2] = -1

    def run(query, idx):
        out = torch.full((R, H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((R, H), 7.0, device=DEV)
        call(query, torch.as_tensor(idx, device=DEV), out, lse)
        torch.cuda.synchronize()
        return out, lse

    want, want_lse = run(q, clean)
    assert want.isfinite().all() and (want_lse.isfinite() | (want_lse == -float("inf"))).all()
    # a NaN row among row 0's keys: in its first tile, in the middle, as the last key; alone
    for at in sorted({0, K // 2, K - 1}):
        idx = clean.copy()
        idx[0, at] = BAD
        out, lse = run(q, idx)
        assert out[0].isnan().all() and lse[0].isnan().all(), at
        assert torch.equal(out[1:], want[1:]) and torch.equal(lse[1:], want_lse[1:])
    idx = np.full_like(clean, -1)
    idx[0, K - 1] = BAD
    out, lse = run(q, idx)
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert not out[1:].any() and (lse[1:] == -float("inf")).all()
    # a NaN in one head of q
    spoilt = q.clone()
    spoilt[1, H // 2, 570] = float("nan")
    out, lse = run(spoilt, clean)
    assert out[1, H // 2].isnan().all() and lse[1, H // 2].isnan()
    keep = torch.ones((R, H), dtype=torch.bool, device=DEV)
    keep[1, H // 2] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
