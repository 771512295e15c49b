"""The scales that the attention over q8 rows refuses, on the host (the calls
that pass this check go on to the next one, a missing q)."""
import ctypes
import math

import pytest
import torch

import __graft_entry__ as G


def _call(scale):
    import hisparse_top_sparse_gb300 as hs
    L = hs.lib()
    rc = L.hs_sparse_attn_decode_q8(None, None, 0, None, 1, 8, 0, ctypes.c_float(scale), None, None, None, 0, None, None)
    return rc, L.hs_last_error_string()


def test_scales_out_of_range_are_refused():
    G.build()
    import hisparse_top_sparse_gb300 as hs
    # 3e38 * log2(e) is no float: scores of 0 would have come out NaN
    for scale in (3e38, math.inf, math.nan, -1e-30, -math.inf):
        rc, why = _call(scale)
        assert rc == hs.HS_ERR_INVALID_ARG and b"scale" in why, (scale, why)
    for scale in (0.0, 1e-45, 1.0, 2.0 ** 127):
        rc, why = _call(scale)
        assert rc == hs.HS_ERR_INVALID_ARG and b"NULL" in why, (scale, why)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [128, 16])
def test_the_largest_scale(H):
    """Scores of 0 weigh all keys alike at every scale that is taken."""
    import hisparse_top_sparse_gb300 as hs
    G.build()
    g = torch.Generator().manual_seed(3)
    rows = (torch.randint(-7, 8, (64, 576), generator=g) * 0.5).to(torch.bfloat16).cuda()   # exact in a q8 row
    cache = torch.zeros((64, 656), dtype=torch.uint8, device="cuda")
    hs.hs_quant_rows(rows, cache)
    q = torch.zeros((2, H, 576), dtype=torch.bfloat16, device="cuda")
    idx = torch.arange(64, dtype=torch.int32, device="cuda").repeat(2, 1)
    want = rows[:, :512].double().mean(0).cpu()            # sums of halves, exact; rounded once to bf16
    for scale in (0.0, 1e-45, 2.0 ** 127):
        out = torch.full((2, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((2, H), float("nan"), device="cuda")
        hs.hs_sparse_attn_decode_q8(q, cache, idx, scale, out, lse=lse)
        assert torch.equal(out.cpu(), want.to(torch.bfloat16).expand(2, H, 512))
        assert ((lse.cpu().double() - math.log(64)).abs() <= 2.0 ** -20).all()
