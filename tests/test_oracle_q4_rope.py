"""Pins of the oracle's 4-bit rows and rotary positions, the library's host
side of the frequencies, and the refusals of the calls that need no GPU."""
import ctypes
import math

import numpy as np
import pytest

import __graft_entry__ as G
from oracle import hs_oracle as O


def test_q4_rows_by_hand():
    x = np.zeros((1, 576))
    # scale 1 (byte 16 * 8): every level, and the middles, which go to the even code
    x[0, :16] = [6, 0.5, -1, 1.5, 2, 3, -4, 0, 0.25, 0.75, 1.25, 1.75, 2.5, -3.5, 5, -0.25]
    x[0, 16:18] = [6.001, 6.75]                     # the scale above 1: 9 / 8 exactly
    x[0, 512:] = np.arange(64)
    r = O.q4_quantise(x)
    assert r.shape == (1, 416) and r[0, 384] == 128 and r[0, 385] == 129 and r[0, 386] == 0
    # dims 0, 2 | 4, 6 | 1, 3 | 5, 7 of the first eight: codes 7 1 10 3 4 5 14 0
    assert list(r[0, :4]) == [7 | 10 << 4, 4 | 14 << 4, 1 | 3 << 4, 5]
    v = O.q4_values(r)[0]
    assert list(v[:8]) == [6, 0.5, -1, 1.5, 2, 3, -4, 0]
    assert list(v[8:16]) == [0, 1, 1, 2, 2, -4, 4, 0]
    assert v[16] == 6.75 and v[17] == 6.75
    assert np.array_equal(v[512:], np.arange(64))


def test_q4_scales_are_the_smallest_that_reach_and_errors_within_the_bound():
    g = np.random.default_rng(1)
    x = (g.standard_normal((60, 576)) * np.exp(g.standard_normal((60, 576)) * 2)).astype(np.float32).astype(np.float64)
    r = O.q4_quantise(x)
    v = O.q4_values(r)
    b = r[:, 384:].astype(int)
    most = np.abs(x[:, :512]).reshape(60, 32, 16).max(2)
    assert (6 * O.Q4_SCALES[b] >= most).all() and (6 * O.Q4_SCALES[b - 1] < most).all()
    bound = np.maximum(np.abs(x[:, :512]), np.repeat(O.Q4_SCALES[b], 16, 1)) / 4
    assert (np.abs(v[:, :512] - x[:, :512]) <= bound).all()
    assert np.array_equal(O.bf16_bits_to_f64(O.f64_to_bf16_bits(v)), v)      # every value is a bf16 number
    assert np.array_equal(O.q4_quantise(v), r) or (O.q4_values(O.q4_quantise(v)) == v).all()


def test_q4_special_values():
    x = np.zeros((2, 576))
    x[0, 0], x[0, 1], x[0, 16], x[0, 32] = np.nan, 3.0, np.inf, -np.inf
    x[0, 48], x[0, 49] = 1e30, -1.0
    x[0, 64] = 1e-30
    r = O.q4_quantise(x)
    v = O.q4_values(r)
    assert np.isnan(v[0, :48]).all() and (r[0, 384:387] == 255).all()
    assert v[0, 48] == 6 * 1.75 * 2.0 ** 15 and v[0, 49] == 0 and r[0, 387] == 254
    assert v[0, 64] == 0 and r[0, 388] == 0
    assert not O.q4_values(np.zeros((1, 416), np.uint8)).any()


def test_rope_by_hand():
    quarter = 1 << 62                                # a quarter of a turn a position
    x = np.arange(1.0, 9).reshape(1, 1, 8)
    y = O.rope_rows(x, [1], [quarter, 0], rot_off=2, half=False)
    assert np.allclose(y[0, 0], [1, 2, -4, 3, 5, 6, 7, 8])
    y = O.rope_rows(x, [1], [quarter, 0], rot_off=2, half=True, factor=2.0)
    assert np.allclose(y[0, 0], [1, 2, -10, 8, 6, 12, 7, 8])
    # a whole number of turns at any position; three quarters is minus a quarter
    assert np.allclose(O.rope_rows(x, [4 * 10 ** 8], [quarter], rot_off=0)[0, 0], x[0, 0])
    assert np.allclose(O.rope_rows(x, [3], [quarter]), O.rope_rows(x, [1], [quarter], inverse=True))
    # relative positions: the product of a query at p and a key at k goes by p - k
    g = np.random.default_rng(0)
    w, _ = O.rope_freqs(16)
    f = [round(v / (2 * math.pi) * 2 ** 64) for v in w]
    q, k = g.standard_normal((1, 1, 16)), g.standard_normal((1, 1, 16))
    dots = [(O.rope_rows(q, [100003 + s], f) * O.rope_rows(k, [99990 + s], f)).sum() for s in (0, 77)]
    assert abs(dots[0] - dots[1]) < 1e-9


def _lib():
    G.build()
    import hisparse_top_sparse_gb300 as hs
    return hs


@pytest.mark.parametrize("rot,kw", [
    (64, {}), (2, {}), (128, dict(base=500000.0)), (64, dict(scaling="linear", scale=8.0)),
    (64, dict(scaling="ntk", scale=4.0)), (64, dict(scaling="yarn", scale=40.0, context=4096)),
    (32, dict(scaling="yarn", scale=16.0, context=8192, fast=16.0, slow=2.0)),
    (64, dict(scaling="yarn", scale=2.0, context=3.0)), (6, dict(scaling="yarn", scale=1.0, context=1e6))])
def test_freqs_against_the_definition(rot, kw):
    hs = _lib()
    code = dict(plain=hs.HS_ROPE_PLAIN, linear=hs.HS_ROPE_LINEAR, ntk=hs.HS_ROPE_NTK, yarn=hs.HS_ROPE_YARN)
    freqs, factor = hs.hs_rope_freqs(rot, **dict(kw, scaling=code[kw.get("scaling", "plain")]))
    w, f = O.rope_freqs(rot, **kw)
    got = freqs.numpy().astype(np.float64) * (2 * math.pi / 2.0 ** 64)
    # a power, a logarithm and a few products in 64 bits, each within some units of 2^-53; the
    # power multiplies its argument's error by its logarithm (below 14)
    assert (np.abs(got - w) <= w * 2.0 ** -46 + 2 * math.pi * 2.0 ** -64).all()
    assert abs(factor - f) <= 2.0 ** -23 * f


def test_freqs_refusals():
    hs = _lib()
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=64, base=1.0), dict(rot_dim=64, base=float("nan")),
               dict(rot_dim=64, scaling=4), dict(rot_dim=64, scaling=1, scale=0.5), dict(rot_dim=2, scaling=2, scale=2.0),
               dict(rot_dim=64, scaling=3, scale=2.0), dict(rot_dim=64, scaling=3, scale=2.0, context=4096, fast=1.0, slow=2.0),
               dict(rot_dim=64, scaling=3, scale=float("inf"), context=4096), dict(rot_dim=1 << 17)):
        with pytest.raises(hs.HisparseError):
            hs.hs_rope_freqs(**kw)


def test_call_refusals_without_a_gpu():
    hs = _lib()
    L = hs.lib()
    bad, p16 = hs.HS_ERR_INVALID_ARG, ctypes.c_void_p(16)
    f = ctypes.c_float

    def quant(src=p16, dt=hs.HS_LOGITS_BF16, stride=576, rows=4, dst=p16, dst_rows=4, ss=None, ds=None, n=4, st=None):
        return L.hs_quant_rows_q4(src, dt, stride, rows, dst, dst_rows, ss, ds, n, st, None)

    def dequant(src=p16, rows=4, dst=p16, dt=hs.HS_LOGITS_BF16, stride=576, dst_rows=4, ss=None, ds=None, n=4, st=None):
        return L.hs_dequant_rows_q4(src, rows, dst, dt, stride, dst_rows, ss, ds, n, st, None)

    for call in (quant, dequant):
        assert call(n=0) == hs.HS_OK
        for kw in (dict(dt=7), dict(n=-1), dict(rows=-1), dict(dst_rows=-1), dict(stride=575), dict(stride=577),
                   dict(src=None), dict(dst=None), dict(src=ctypes.c_void_p(24)), dict(dst=ctypes.c_void_p(20)),
                   dict(ss=ctypes.c_void_p(2)), dict(ds=ctypes.c_void_p(6)), dict(st=ctypes.c_void_p(3))):
            assert call(**kw) == bad, kw

    def attn(q=p16, kv=p16, n=4, idx=p16, R=1, H=1, K=1, scale=1.0, out=p16, lse=None, ws=None, size=0, st=None):
        return L.hs_sparse_attn_decode_q4(q, kv, n, idx, R, H, K, f(scale), out, lse, ws, size, st, None)

    assert attn(R=0) == hs.HS_OK
    for kw in (dict(R=-1), dict(H=0), dict(H=1025), dict(K=-1), dict(n=-1), dict(q=None), dict(kv=None), dict(idx=None),
               dict(out=None), dict(q=ctypes.c_void_p(8)), dict(kv=ctypes.c_void_p(8)), dict(out=ctypes.c_void_p(8)),
               dict(scale=-1.0), dict(scale=2.0 ** 101), dict(scale=float("nan")), dict(ws=ctypes.c_void_p(8)),
               dict(idx=ctypes.c_void_p(18)), dict(lse=ctypes.c_void_p(2)), dict(st=ctypes.c_void_p(1))):
        assert attn(**kw) == bad, kw

    def rope(src=p16, srow=64, shead=64, srows=4, dst=p16, drow=64, dhead=64, drows=4, dt=hs.HS_LOGITS_BF16, ss=None,
             ds=None, pos=p16, n=4, heads=1, dim=64, off=0, rot=64, layout=0, freqs=p16, factor=1.0, st=None):
        return L.hs_rope_rows(src, srow, shead, srows, dst, drow, dhead, drows, dt, ss, ds, pos, n, heads, dim, off, rot,
                              layout, freqs, f(factor), 0, st, None)

    assert rope(n=0) == hs.HS_OK
    for kw in (dict(dt=2), dict(layout=2), dict(n=-1), dict(srows=-1), dict(drows=-1), dict(heads=0), dict(heads=65536),
               dict(dim=1, rot=2), dict(rot=63), dict(rot=0), dict(rot=66), dict(off=-2), dict(off=2), dict(dim=65537),
               dict(srow=-1), dict(dhead=-1), dict(drow=(1 << 40) + 1), dict(factor=float("nan")), dict(factor=float("inf")),
               dict(src=None), dict(dst=None), dict(pos=None), dict(freqs=None), dict(freqs=ctypes.c_void_p(20)),
               dict(src=ctypes.c_void_p(17)), dict(dst=ctypes.c_void_p(18), dt=hs.HS_LOGITS_F32),
               dict(pos=ctypes.c_void_p(18)), dict(ss=ctypes.c_void_p(2)), dict(ds=ctypes.c_void_p(2)),
               dict(st=ctypes.c_void_p(2)),
               dict(drow=63), dict(heads=2, drow=128, dhead=63), dict(heads=2, drow=127, dhead=64),
               dict(heads=2, drow=64, dhead=255),             # rows or heads of dst share elements
               dict(heads=2, drow=64, dhead=1 << 40, drows=1 << 62), dict(heads=65535, drow=1 << 40, dhead=1 << 40, dim=64)):
        assert rope(**kw) == bad, kw
    assert rope(heads=40000, dim=40000, dhead=40000, drow=40000 * 40000, n=4) == hs.HS_ERR_UNSUPPORTED


def test_the_bindings_short_way_leaves_to_the_long_one_what_it_does_not_take():
    import torch
    hs = _lib()
    hs.lib()
    if hs._native is None:
        pytest.skip("no headers of this Python: the native module is not built")
    N, addr = hs._native, hs._ADDR
    x, c = torch.zeros((4, 576)), torch.zeros((4, 416), dtype=torch.uint8)
    pos, freqs = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    q, idx = torch.zeros((2, 3, 576), dtype=torch.bfloat16), torch.zeros((2, 5), dtype=torch.int32)
    out = torch.zeros((2, 3, 512), dtype=torch.bfloat16)
    for _ in range(3):
        # tensors of the host (whatever the current device is), and what are no tensors
        assert N.quant(addr["hs_quant_rows_q4"], 416, x, c, None, None, None, 0) is None
        assert N.dequant(addr["hs_dequant_rows_q4"], 416, c, x, pos, None, None, None) is None
        assert N.attend(addr["hs_sparse_attn_decode_q4"], 416, q, c, idx, 1.0, out, None, None, None, 0) is None
        assert N.rope(addr["hs_rope_rows"], x, x, pos, freqs, 1.0, 0, 0, False, None, None, None, 0) is None
        assert N.quant(addr["hs_quant_rows_q4"], 416, "x", 7, None, None, None, 0) is None
        assert N.rope(addr["hs_rope_rows"], None, x, 3, [], "f", 0, 0, 1, None, None, None, 0) is None
        assert N.quant() is None and N.attend(1, 2) is None
    with pytest.raises(ValueError):
        hs.hs_quant_rows_q4(x, c)
    with pytest.raises(TypeError):
        N.setup(1)
