"""Rows quantised and read back in numbers that take every warp through its loop
several times, the slots of the next rows loaded ahead: bytes and values of every
row, q4 and q8, against the oracle."""
import numpy as np
import pytest
import torch

from oracle import hs_oracle as O
from gpu_util import lib, np_
from test_gpu_q4 import _check_bytes, _f64, _t

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _slots(g, n, rows, most):
    """n slots: of `rows` rows, distinct where `most` is None; some no entry, some past
    the rows."""
    s = (g.permutation(rows)[:n] if most is None else g.integers(0, most, size=n)).astype(np.int32)
    s[3::17] = -1
    s[5::1009] = rows
    s[6::2003] = np.iinfo(np.int32).max
    return s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,n", [("q4", 20011), ("q4", 60001), ("q8", 20011)])
def test_rows_of_many_turns(fmt, n, dtype):
    hs = lib()
    if fmt == "q4":
        row, quant, dequant, encode, decode = 416, hs.hs_quant_rows_q4, hs.hs_dequant_rows_q4, O.q4_quantise, O.q4_values
    else:
        row, quant, dequant, encode, decode = 656, hs.hs_quant_rows, hs.hs_dequant_rows, O.q8_quantise, O.q8_values
    # rows in flight: two of a bf16 row's warp, one of an f32 row's, eight warps a block, four blocks an SM
    turn = 32 * torch.cuda.get_device_properties(0).multi_processor_count * (2 if dtype == torch.bfloat16 else 1)
    assert n > 2 * turn and n % turn
    g = np.random.default_rng(n + row)
    src_rows, rows = n + 5, n + 301
    x = g.standard_normal((src_rows, 576), dtype=np.float32) * np.exp(g.standard_normal((1, 576), dtype=np.float32))
    src = torch.as_tensor(x).to(dtype).to(DEV)
    cache = torch.full((rows, row), 0xA5, dtype=torch.uint8, device=DEV)
    s, d = _slots(g, n, src_rows, src_rows), _slots(g, n, rows, None)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    quant(src, cache, src_slots=_t(s), dst_slots=_t(d), status=st)
    assert int(st.item()) == hs.HS_STATUS_INDEX
    ok = (s >= 0) & (d >= 0) & (s < src_rows) & (d < rows)
    whole = encode(_f64(src))
    want = np.full((rows, row), 0xA5, np.uint8)
    want[d[ok]] = whole[s[ok]]
    got = np_(cache)
    held = np.zeros(rows, bool)
    held[d[ok]] = True
    assert np.array_equal(got[~held], want[~held])
    if fmt == "q4":
        _check_bytes(got[held], want[held])
    else:
        assert np.array_equal(got[held], want[held])
    # read back into other slots; the rows' values are the stored bytes'
    s2, d2 = _slots(g, n, rows, rows), _slots(g, n, rows, None)
    s2 = np.where((s2 >= 0) & (s2 < rows), d[ok][s2 % ok.sum()], s2).astype(np.int32)      # rows that were written
    st.zero_()
    back = torch.full((rows, 576), 5.0, dtype=dtype, device=DEV)
    dequant(cache, back, src_slots=_t(s2), dst_slots=_t(d2), status=st)
    assert int(st.item()) == hs.HS_STATUS_INDEX
    ok2 = (s2 >= 0) & (d2 >= 0) & (s2 < rows) & (d2 < rows)
    e = np.full((rows, 576), 5.0)
    e[d2[ok2]] = decode(want[s2[ok2]])
    assert np.array_equal(_f64(back), e)
    # and without lists
    plain = torch.zeros((src_rows, row), dtype=torch.uint8, device=DEV)
    st.zero_()
    quant(src, plain, status=st)
    if fmt == "q4":
        _check_bytes(np_(plain), whole)
    else:
        assert np.array_equal(np_(plain), whole)
    out = torch.zeros((src_rows, 576), dtype=dtype, device=DEV)
    dequant(plain, out, status=st)
    assert np.array_equal(_f64(out), decode(whole)) and int(st.item()) == 0
