"""Pins of the oracle's quantised rows and of its sampled verification, and the
refusals of the calls that need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__ as G
from oracle import hs_oracle as O


def test_e4m3_table_and_rounding_agree_with_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(want), np.isnan(O.E4M3_VALUES))
    ok = ~np.isnan(want)
    assert np.array_equal(want[ok], O.E4M3_VALUES[ok])
    g = np.random.default_rng(0)
    x = np.concatenate([g.standard_normal(4000) * 100, g.standard_normal(2000) * 0.01,
                        O._E4M3_MIDS, -O._E4M3_MIDS, O._E4M3_MAGS])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = O.e4m3_encode(x.astype(np.float64))
    zero = O.E4M3_VALUES[got] == 0
    assert np.array_equal(got[~zero], want[~zero]) and not O.E4M3_VALUES[want[zero]].any()


def test_q8_rows_by_hand():
    x = np.zeros((1, 576))
    x[0, 0], x[0, 1], x[0, 2] = 448.0, -1.0, 2.0 ** -9          # e = 0: held exactly
    x[0, 32], x[0, 33] = 448.5, 17.0                             # e = 1: 448 -> 448/2, ...
    x[0, 512:] = np.arange(64)
    r = O.q8_quantise(x)
    assert r.shape == (1, 656) and r[0, 640] == 127 and r[0, 641] == 128 and r[0, 642] == 15
    v = O.q8_values(r)[0]
    assert v[0] == 448 and v[1] == -1 and v[2] == 2.0 ** -9
    # 224.25 -> 224; 8.5 lies between the codes of 8 and 9 and goes to the even one
    assert v[32] == 448 and v[33] == 16
    assert np.array_equal(v[512:], np.arange(64))


def test_q8_error_is_half_a_step_and_values_are_bf16():
    g = np.random.default_rng(1)
    x = (g.standard_normal((50, 576)) * np.exp(g.standard_normal((50, 576)) * 3)).astype(np.float32)
    r = O.q8_quantise(x.astype(np.float64))
    v = O.q8_values(r)
    e = np.repeat(r[:, 640:].astype(np.float64) - 127, 32, axis=1)
    bound = np.maximum(np.abs(x[:, :512]) * 2.0 ** -4, 2.0 ** (e - 10))
    assert (np.abs(v[:, :512] - x[:, :512]) <= bound).all()
    assert np.array_equal(O.bf16_bits_to_f64(O.f64_to_bf16_bits(v)), v)


def test_q8_special_values():
    x = np.zeros((1, 576))
    x[0, 0], x[0, 1] = np.nan, 3.0
    x[0, 32], x[0, 33] = np.inf, 1.0
    x[0, 64] = -np.inf
    v = O.q8_values(O.q8_quantise(x))[0]
    assert math.isnan(v[0]) and v[1] == 3.0
    assert v[32] == np.inf and v[33] == 0.0 and v[64] == -np.inf
    assert (O.q8_values(np.zeros((2, 656), np.uint8)) == 0).all()


def _step(l, T, x, q, u, E):
    a, t, lp, _ = O.verify_sample(np.array([l]), [T], np.array([x]), q, np.array([u]), np.array([E]))
    return int(a[0]), int(t[0]), lp[0]


def test_verify_sample_by_hand():
    ln = math.log
    # p = (1/2, 1/4, 1/4) twice; the draft 1 has q = 1/2: accepted below u = 1/2
    l = [[ln(2), 0.0, 0.0]] * 2
    q = np.array([[[0.25, 0.5, 0.25]]])
    assert _step(l, 1.0, [1], q, [0.49], [1, 1, 1])[:2] == (1, 0)
    # refused: w = (1/4, 0, 0)
    m, t, lp = _step(l, 1.0, [1], q, [0.5], [100.0, 1e-3, 1e-3])
    assert (m, t) == (0, 0) and abs(lp[0] - ln(0.5)) < 1e-12 and lp[1] == 0
    # a sure draft is accepted below u = p and not drawn after a refusal
    assert _step(l, 1.0, [0], None, [0.49], [1, 1, 9])[0] == 1
    assert _step(l, 1.0, [0], None, [0.51], [1e-9, 1, 0.5])[:2] == (0, 2)
    # the race past the last draft, ties to the lowest index
    assert _step(l, 1.0, [0], None, [0.0], [2.0, 1.0, 1.0])[:2] == (1, 0)
    # greedy, masked rows, bad drafts
    assert _step([[0, 3, 3], [5, 1, 1]], 0.0, [1], None, [0.9], [1, 1, 1])[:2] == (1, 0)
    assert _step([[-np.inf] * 3] * 2, 1.0, [1], None, [0.0], [1, 1, 1])[:2] == (0, -1)
    assert _step(l, 1.0, [7], None, [0.0], [1, 1, 1])[0] == 0
    # nothing left past the draft's figures: the target's own probabilities
    assert _step(l, 1.0, [2], np.ones((1, 1, 3)), [0.9], [1, 1, 0.1])[:2] == (0, 2)


def test_verify_sample_is_distributed_as_the_target():
    """The first token given, accepted draft or drawn, follows p_0."""
    g = np.random.default_rng(3)
    V, n = 5, 20000
    l = g.standard_normal((1, 2, V)).repeat(n, 0)
    q = np.exp(g.standard_normal(V))
    q /= q.sum()
    x = g.choice(V, size=(n, 1), p=q)
    a, t, _, _ = O.verify_sample(l, np.ones(n), x, np.broadcast_to(q, (n, 1, V)), g.random((n, 1)),
                                 g.exponential(size=(n, V)))
    first = np.where(a == 1, x[:, 0], t)
    p = np.exp(l[0, 0]) / np.exp(l[0, 0]).sum()
    got = np.bincount(first, minlength=V) / n
    assert (np.abs(got - p) <= 5 * np.sqrt(p * (1 - p) / n)).all()


def test_refusals_without_a_gpu():
    G.build()
    import hisparse_top_sparse_gb300 as hs
    L = hs.lib()
    P = ctypes.c_void_p
    bad = hs.HS_ERR_INVALID_ARG

    def quant(src=P(16), dt=1, stride=576, rows=4, dst=P(16), drows=4, n=1):
        return L.hs_quant_rows(src, dt, stride, rows, dst, drows, None, None, n, None, None)

    def dequant(src=P(16), rows=4, dst=P(16), dt=1, stride=576, drows=4, n=1):
        return L.hs_dequant_rows(src, rows, dst, dt, stride, drows, None, None, n, None, None)

    for f in (quant, dequant):
        assert f(dt=2) == bad and f(stride=575) == bad and f(stride=577) == bad
        assert f(rows=-1) == bad and f(drows=-1) == bad and f(n=-1) == bad
        assert f(src=None) == bad and f(dst=None) == bad and f(src=P(8)) == bad and f(dst=P(8)) == bad
        assert f(src=None, dst=None, n=0) == hs.HS_OK
    assert b"16-byte" in L.hs_last_error_string()

    def attn(q=P(16), kv=P(16), rows=4, idx=P(16), R=1, H=1, K=0, scale=1.0, out=P(16), ws=None):
        return L.hs_sparse_attn_decode_q8(q, kv, rows, idx, R, H, K, ctypes.c_float(scale), out, None,
                                          ws, 0, None, None)

    assert attn(H=0) == bad and attn(H=1025) == bad and attn(R=-1) == bad and attn(K=-1) == bad
    assert attn(rows=-1) == bad and attn(q=None) == bad and attn(out=None) == bad
    assert attn(K=1, idx=None) == bad and attn(K=1, kv=None) == bad
    assert attn(q=P(8)) == bad and attn(kv=P(8)) == bad and attn(out=P(8)) == bad and attn(ws=P(8)) == bad
    assert attn(scale=float("nan")) == bad and attn(scale=-0.5) == bad and attn(scale=float("inf")) == bad
    assert attn(R=0) == hs.HS_OK

    def sample(l=P(16), dt=0, B=1, d=1, V=8, t=P(16), x=P(16), u=P(16), e=P(16), a=P(16), n=P(16), q=None):
        return L.hs_verify_sample(l, dt, B, d, V, t, x, q, u, e, a, n, None, None, None)

    assert sample(B=0) == bad and sample(d=-1) == bad and sample(d=256) == bad and sample(V=0) == bad
    assert sample(V=(1 << 30) + 1) == bad and sample(dt=2) == bad
    for k in "ltxuean":
        assert sample(**{k: None}) == bad
    assert sample(l=P(18)) == bad and sample(dt=1, l=P(17)) == bad and sample(q=P(18)) == bad
    for k in "txueanq":
        assert sample(**{k: P(18)}) == bad
    for lp, st in ((P(18), None), (None, P(18))):
        assert L.hs_verify_sample(P(16), 0, 1, 1, 8, P(16), P(16), None, P(16), P(16), P(16), P(16), lp, st,
                                  None) == bad
        assert L.hs_sparse_attn_decode_q8(P(16), P(16), 4, P(16), 1, 1, 1, ctypes.c_float(1.0), P(16), lp,
                                          None, 0, st, None) == bad
    for ss, ds, st in ((P(18), None, None), (None, P(18), None), (None, None, P(18))):
        assert L.hs_quant_rows(P(16), 1, 576, 4, P(16), 4, ss, ds, 1, st, None) == bad
        assert L.hs_dequant_rows(P(16), 4, P(16), 1, 576, 4, ss, ds, 1, st, None) == bad
    assert L.hs_verify_sample_finalize(None, P(16), 0, 1, 0, 8, P(16), None, None, None, P(16), P(16),
                                       None, P(16), P(16), P(16), None, None) == bad


def test_binding_refuses_wrong_tensors():
    G.build()
    import hisparse_top_sparse_gb300 as hs
    x = torch.zeros((4, 576), dtype=torch.bfloat16)
    c = torch.zeros((4, 656), dtype=torch.uint8)
    for f, args in ((hs.hs_quant_rows, (x, c)), (hs.hs_dequant_rows, (c, x))):
        with pytest.raises(ValueError):
            f(*args)                                   # neither CUDA nor pinned
    with pytest.raises((ValueError, TypeError)):
        hs.hs_quant_rows(None, c)
    with pytest.raises(ValueError):
        hs.hs_sparse_attn_decode_q8(torch.zeros((1, 2, 575), dtype=torch.bfloat16), c,
                                    torch.zeros((1, 1), dtype=torch.int32), 1.0, None)
    with pytest.raises(TypeError):
        hs.hs_verify_sample(torch.zeros((1, 2, 3), dtype=torch.float16), None, None, None, None, None,
                            None, None)
