"""GPU parity of the quantised latent rows (hs_quant_rows, hs_dequant_rows) and
of the attention over them (hs_sparse_attn_decode_q8): bytes and values
bit-exact against the oracle, attention within bounds derived from its
roundings, and bit-identical to hs_sparse_attn_decode over the same values."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import workloads as W
from oracle import hs_oracle as O
from gpu_util import lib, np_

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _t(a):
    return torch.as_tensor(np.ascontiguousarray(a), device=DEV)


def _rows(g, n, dtype, width=576):
    x = g.standard_normal((n, width)) * np.exp(g.standard_normal((n, width)) * 2)
    return torch.as_tensor(x.astype(np.float32)).to(dtype)


def _f64(x):
    return x.detach().cpu().double().numpy()


def _check_bytes(got, want):
    nan = (want[:, :512] & 0x7F) == 0x7F
    assert np.array_equal((got[:, :512] & 0x7F) == 0x7F, nan)
    assert np.array_equal(got[:, :512][~nan], want[:, :512][~nan])
    r = O.bf16_bits_to_f64(np.ascontiguousarray(want[:, 512:640]).view(np.uint16))
    s = O.bf16_bits_to_f64(np.ascontiguousarray(got[:, 512:640]).view(np.uint16))
    assert np.array_equal(r, s, equal_nan=True)
    assert np.array_equal(got[:, 640:], want[:, 640:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,width,offset", [(1, 576, 0), (7, 640, 64), (300, 1152, 8), (2500, 584, 8)])
def test_quant_rows_bytes(dtype, n, width, offset):
    hs = lib()
    g = np.random.default_rng(n + width)
    wide = _rows(g, n, dtype, width).to(DEV)
    src = wide[:, offset:offset + 576]
    rows = n + 11
    cache = torch.full((rows, 656), 0xA5, dtype=torch.uint8, device=DEV)
    slots = g.permutation(rows)[:n].astype(np.int32)
    slots[::5] = -1
    hs.hs_quant_rows(src, cache, dst_slots=_t(slots))
    want = np.full((rows, 656), 0xA5, np.uint8)
    keep = slots >= 0
    if keep.any():
        want[slots[keep]] = O.q8_quantise(_f64(src)[keep])
    got = np_(cache)
    held = np.zeros(rows, bool)
    held[slots[keep]] = True
    assert np.array_equal(got[~held], want[~held])     # rows without an entry stay as they were
    if keep.any():
        _check_bytes(got[held], want[held])


def test_quant_rows_special_values():
    hs = lib()
    big = float(torch.finfo(torch.float32).max)
    x = torch.zeros((6, 576))
    x[0, ::32] = torch.tensor([0.0, 448, 448.001, 1e-38, 1e-45, 2.0 ** -121, 2.0 ** -112, 449, 447.9,
                               2.0 ** 127, 3.0e38, 3.4e38, -448, 224.0001, -0.0, 5, 6, 7])
    x[1, 0], x[1, 1] = float("nan"), 3.0
    x[1, 32], x[1, 33], x[1, 64] = float("inf"), 1.0, -float("inf")
    x[1, 575], x[1, 574] = float("nan"), float("inf")
    x[2, :512] = torch.linspace(-448, 448, 512)            # every code's neighbourhood
    x[3, :512] = (torch.arange(512) % 256).to(torch.uint8).view(torch.float8_e4m3fn).float().nan_to_num(1.0)
    x[4, :32] = big
    x[5, :512] = 2.0 ** torch.arange(-256, 256).float().clamp(-149, 127)
    for dtype in (torch.float32, torch.bfloat16):
        src = x.to(dtype)
        cache = torch.empty((6, 656), dtype=torch.uint8, device=DEV)
        hs.hs_quant_rows(src.to(DEV), cache)
        want = O.q8_quantise(_f64(src))
        _check_bytes(np_(cache), want)
        for out_t in (torch.float32, torch.bfloat16):
            back = torch.empty((6, 576), dtype=out_t, device=DEV)
            hs.hs_dequant_rows(cache, back)
            assert np.array_equal(_f64(back), O.q8_values(want), equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequant_rows_every_code_and_exponent(dtype):
    hs = lib()
    g = np.random.default_rng(4)
    rows = np.zeros((300, 656), np.uint8)
    rows[:, :512] = (np.arange(512) + np.arange(300)[:, None] * 7) % 256
    rows[:, 512:640] = g.integers(0, 127, (300, 128))       # finite bf16 values
    rows[:233, 640:] = np.arange(15, 248)[:, None]
    rows[233:, 640:] = g.integers(15, 248, (67, 16))
    rows[299] = 0                                           # a row never written
    want = O.q8_values(rows)
    slots = g.integers(-1, 300, size=1000).astype(np.int32)
    slots[:300] = np.arange(300)
    dst = g.permutation(1100)[:1000].astype(np.int32)
    dst[3::50] = -1
    wide = torch.full((1100, 640), 7.0, dtype=dtype, device=DEV)
    hs.hs_dequant_rows(_t(rows), wide[:, 64:], src_slots=_t(slots), dst_slots=_t(dst))
    e = np.full((1100, 640), 7.0)
    keep = (slots >= 0) & (dst >= 0)
    e[dst[keep], 64:] = want[slots[keep]]
    assert np.array_equal(_f64(wide), e, equal_nan=True)


def test_row_calls_report_bad_slots_and_leave_the_rest():
    hs = lib()
    g = np.random.default_rng(5)
    src = _rows(g, 10, torch.bfloat16).to(DEV)
    cache = torch.zeros((12, 656), dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    s = np.array([0, 10, 3, -1, 5], np.int32)
    d = np.array([2, 3, 12, 4, 5], np.int32)
    hs.hs_quant_rows(src, cache, src_slots=_t(s), dst_slots=_t(d), status=st)
    assert int(st.item()) == hs.HS_STATUS_INDEX
    want = np.zeros((12, 656), np.uint8)
    want[[2, 5]] = O.q8_quantise(_f64(src)[[0, 5]])
    assert np.array_equal(np_(cache), want)
    st.zero_()
    back = torch.full((4, 576), 9.0, device=DEV)
    hs.hs_dequant_rows(cache, back, src_slots=_t(np.array([2, 12, 5], np.int32)),
                       dst_slots=_t(np.array([1, 0, 4], np.int32)), status=st)
    assert int(st.item()) == hs.HS_STATUS_INDEX
    e = np.full((4, 576), 9.0)
    e[1] = O.q8_values(want[2:3])[0]
    assert np.array_equal(_f64(back), e)
    # nothing to do
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    hs.hs_quant_rows(src, cache, src_slots=none, dst_slots=none)
    with pytest.raises(ValueError):
        hs.hs_quant_rows(src, cache[:4])                   # ten rows into four
    with pytest.raises(ValueError):
        hs.hs_quant_rows(src, cache, src_slots=_t(s), dst_slots=_t(d[:3]))
    with pytest.raises(ValueError):
        hs.hs_quant_rows(src.t().contiguous().t(), cache)
    with pytest.raises(hs.HisparseError):
        hs.hs_quant_rows(torch.zeros((4, 577), dtype=torch.bfloat16, device=DEV)[:, 1:], cache)


def test_quant_rows_to_host_and_back():
    """Rows quantised into a page-locked host cache (a backup that shrinks),
    then read back from it."""
    hs = lib()
    g = np.random.default_rng(6)
    src = _rows(g, 500, torch.bfloat16).to(DEV)
    host = torch.zeros((700, 656), dtype=torch.uint8, pin_memory=True)
    d = g.permutation(700)[:500].astype(np.int32)
    hs.hs_quant_rows(src, host, dst_slots=_t(d))
    back = torch.zeros((500, 576), dtype=torch.bfloat16, device=DEV)
    hs.hs_dequant_rows(host, back, src_slots=_t(d))
    torch.cuda.synchronize()
    want = O.q8_quantise(_f64(src))
    assert np.array_equal(host.numpy()[d], want)
    assert np.array_equal(_f64(back), O.q8_values(want))


# ------------------------------------------------------------- attention --

def _cache(g, n):
    """q8 rows of latent-like values, and their values."""
    rows = O.q8_quantise(g.standard_normal((n, 576)) * np.exp(0.5 * g.standard_normal((1, 576))))
    return rows, O.q8_values(rows)


def _indices(g, R, K, n, pad):
    idx = g.integers(0, n, size=(R, K)).astype(np.int32)
    idx[g.random((R, K)) < pad] = -1
    return idx


def _check(out, lse, q, values, idx, scale):
    """Bounds from the roundings: the numerators and the output to bf16 (half
    a step 2^-8 each, the first averaged over the values' magnitudes A), the
    products' sums and the exponentials in f32 (the score of a key is off by at
    most `ds`, its numerator relatively by twice that)."""
    R, H, _ = q.shape
    K = idx.shape[1]
    got, got_lse = _f64(out), _f64(lse)
    for r in range(R):
        keep = idx[r][(idx[r] >= 0) & (idx[r] < len(values))]
        if keep.size == 0:
            assert not got[r].any() and np.isneginf(got_lse[r]).all()
            continue
        k = values[keep]
        s = q[r] @ k.T * scale
        ds = (576 * 2.0 ** -23) * scale * (np.abs(q[r]) @ np.abs(k).T).max()
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        l = p.sum(1, keepdims=True)
        want, A = (p / l) @ k[:, :512], (p / l) @ np.abs(k[:, :512])
        rel = 2 * ds + (K + 64) * 2.0 ** -23
        bound = (A + np.abs(want)) * (2.0 ** -8 * (1 + 2.0 ** -7) + rel) + 1e-30
        assert (np.abs(got[r] - want) <= bound).all(), (np.abs(got[r] - want) / bound).max()
        want_lse = (top + np.log(l))[:, 0]
        assert (np.abs(got_lse[r] - want_lse) <= ds + (K + 64) * 2.0 ** -23 +
                4 * 2.0 ** -23 * np.abs(want_lse)).all()


def _attend(hs, q, cache, idx, scale, ws=None, **kw):
    R, H, _ = q.shape
    out = torch.full((R, H, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((R, H), float("nan"), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    hs.hs_sparse_attn_decode_q8(q, cache, idx, scale, out, lse=lse, workspace=ws, status=st, **kw)
    assert int(st.item()) == 0
    return out, lse


CASES = [(1, 1, 1, 0.0), (3, 16, 5, 0.0), (2, 128, 2048, 0.0), (5, 40, 33, 0.3), (2, 136, 130, 0.1),
         (1, 128, 8192, 0.05), (80, 128, 96, 0.5), (9, 64, 1000, 0.9), (1, 1024, 300, 0.0),
         (4, 128, 127, 0.0), (4, 128, 129, 0.0), (7, 16, 2048, 0.1), (320, 8, 100, 0.3), (1, 16, 8192, 0.0),
         (2, 1, 1528, 0.5), (40, 15, 700, 0.97), (3, 17, 300, 0.0), (400, 16, 1, 0.1), (6, 4, 257, 0.0)]


@pytest.mark.parametrize("R,H,K,pad", CASES)
@pytest.mark.parametrize("workspace", [0, 1 << 20, 32 << 20])
def test_attention_against_the_oracle(R, H, K, pad, workspace):
    hs = lib()
    g = np.random.default_rng(R * 10007 + H * 101 + K)
    rows, values = _cache(g, 700)
    idx = _indices(g, R, K, 700, pad)
    if R > 2:
        idx[1] = -1                                        # a row without keys
        idx[2, 0] = 700                                    # skipped: past the cache
    q = torch.as_tensor(g.standard_normal((R, H, 576)).astype(np.float32)).to(torch.bfloat16)
    scale = 1 / 24
    ws = torch.full((workspace,), 0xFF, dtype=torch.uint8, device=DEV) if workspace else None
    out, lse = _attend(hs, q.to(DEV), _t(rows), _t(idx), scale, ws)
    _check(out, lse, _f64(q), values, idx, scale)
    again, lse2 = _attend(hs, q.to(DEV), _t(rows), _t(idx), scale, ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("R,H,K", [(3, 128, 2048), (100, 128, 200), (2, 20, 77)])
def test_attention_equals_the_bf16_call_over_the_same_values(R, H, K):
    """Without a workspace the tiles, their order and their values are those of
    hs_sparse_attn_decode over the rows read back."""
    hs = lib()
    g = np.random.default_rng(R + K)
    rows, values = _cache(g, 3000)
    idx = _t(_indices(g, R, K, 3000, 0.1))
    q = torch.as_tensor(g.standard_normal((R, H, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    cache = _t(rows)
    wide = torch.empty((3000, 576), dtype=torch.bfloat16, device=DEV)
    hs.hs_dequant_rows(cache, wide)
    out, lse = _attend(hs, q, cache, idx, 0.04)
    ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
    hs.hs_sparse_attn_decode(q, wide, idx, 0.04, ref, lse=ref_lse)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("H", [128, 16])
def test_attention_second_pass_and_sharp_logits(H):
    """Scores whose later tiles pass the first ones by more than 2^30."""
    hs = lib()
    g = np.random.default_rng(9)
    x = g.standard_normal((600, 576))
    x[300:] *= 40
    rows = O.q8_quantise(x)
    values = O.q8_values(rows)
    idx = np.arange(600, dtype=np.int32)[None].repeat(3, 0)
    q = torch.as_tensor(g.standard_normal((3, H, 576)).astype(np.float32)).to(torch.bfloat16)
    for ws in (None, torch.empty(32 << 20, dtype=torch.uint8, device=DEV)):
        out, lse = _attend(hs, q.to(DEV), _t(rows), _t(idx), 0.25, ws)
        _check(out, lse, _f64(q), values, idx, 0.25)


@pytest.mark.parametrize("H", [8, 40])
def test_attention_ignores_what_it_does_not_select(H):
    """NaN and infinity in rows that no index names, exact single keys, and
    duplicates counted each time."""
    hs = lib()
    g = np.random.default_rng(10)
    rows, values = _cache(g, 64)
    rows[40:, :512] = 0x7F
    rows[40:, 512:640] = 0xFF
    q = torch.as_tensor(g.standard_normal((2, H, 576)).astype(np.float32)).to(torch.bfloat16)
    idx = np.array([[-1, 7, -1, 64], [3, 3, 5, -7]], np.int32)
    out, lse = _attend(hs, q.to(DEV), _t(rows), _t(idx), 1 / 24)
    _check(out, lse, _f64(q), values, idx, 1 / 24)
    assert torch.equal(out[0].cpu(), torch.as_tensor(values[7, :512]).to(torch.bfloat16).expand(H, 512))
    # a selected NaN row reaches the output in every split
    idx = np.zeros((1, 2048), np.int32)
    idx[0, 2000] = 50
    for ws in (None, torch.empty(32 << 20, dtype=torch.uint8, device=DEV)):
        out, lse = _attend(hs, q[:1].to(DEV), _t(rows), _t(idx), 1 / 24, ws)
        assert out.isnan().all()


def test_attention_in_a_cache_past_4_gib():
    """Row offsets past 32 bits."""
    hs = lib()
    g = np.random.default_rng(11)
    n = (1 << 32) // 656 + 1000
    rows, values = _cache(g, 512)
    cache = torch.zeros((n, 656), dtype=torch.uint8, device=DEV)
    at = np.sort(g.permutation(900)[:512]) + n - 900
    hs_rows = _t(at.astype(np.int64))
    cache[hs_rows] = _t(rows)
    idx = at[g.integers(0, 512, size=(2, 600))].astype(np.int32)
    q = torch.as_tensor(g.standard_normal((2, 128, 576)).astype(np.float32)).to(torch.bfloat16)
    out, lse = _attend(hs, q.to(DEV), cache, _t(idx), 1 / 24, torch.empty(32 << 20, dtype=torch.uint8, device=DEV))
    _check(out, lse, _f64(q), values, np.searchsorted(at, idx).astype(np.int32), 1 / 24)
    # and the row calls at the cache's end
    back = torch.empty((3, 576), device=DEV)
    hs.hs_dequant_rows(cache, back, src_slots=_t(at[-3:].astype(np.int32)))
    assert np.array_equal(_f64(back), values[-3:])


@pytest.mark.parametrize("H", [128, 10])
def test_attention_on_a_side_stream_and_in_graphs(H):
    """Two captured calls, a workspace each, replayed on two streams at once
    over new inputs; the eager call on a side stream."""
    hs = lib()
    g = np.random.default_rng(12)
    rows, _ = _cache(g, 900)
    cache = _t(rows)
    mk = lambda: (torch.as_tensor(g.standard_normal((3, H, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV),
                  _t(_indices(g, 3, 1500, 900, 0.1)))
    ins = [mk(), mk()]
    ws = [torch.empty(32 << 20, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [_attend(hs, q, cache, idx, 1 / 24, w) for (q, idx), w in zip(ins, ws)]
    got = [(torch.empty_like(o), torch.empty_like(l)) for o, l in outs]
    graphs = []
    for i, (q, idx) in enumerate(ins):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            hs.hs_sparse_attn_decode_q8(q, cache, idx, 1 / 24, got[i][0], lse=got[i][1], workspace=ws[i])
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(3):
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for (q, idx), (o, l) in zip(ins, got):
            e, e_l = _attend(hs, q, cache, idx, 1 / 24, ws[0])
            assert torch.equal(o, e) and torch.equal(l, e_l)
        for q, idx in ins:                                  # new inputs in the same places
            nq, ni = mk()
            q.copy_(nq)
            idx.copy_(ni)
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        o, l = _attend(hs, *[ins[0][0], cache, ins[0][1], 1 / 24, ws[0]])
    torch.cuda.synchronize()
    e, e_l = _attend(hs, ins[0][0], cache, ins[0][1], 1 / 24, ws[0])
    assert torch.equal(o, e) and torch.equal(l, e_l)


def test_a_step_over_a_q8_follower_layer():
    """The operators as a step uses them: rows quantised into a follower's
    host pool and step slots, the leader's swap-in, its plan repeated for the
    656-byte rows, attention over the follower through the leader's slot
    table, sampled verify and commit."""
    hs = lib()
    cfg = W.get_config(1)
    req, ri = W.rows_of(cfg)
    hb = W.host_backed_case(cfg, device=DEV, extra_positions=8)
    buf = hs.HsBuffer(cfg.B, cfg.S, cfg.d + 1, hb["max_ctx"], cfg.block_size, hb["hot"], hb["pool"], hb["hbt"])
    ref = O.HotBuffer(cfg.B, cfg.S, cfg.d + 1, hb["max_ctx"], cfg.block_size, hb["hbt_np"], hb["pool"].clone())
    n_pool, n_hot, S_tot = hb["pool"].shape[0], hb["hot"].shape[0], cfg.S + cfg.d + 1
    layer = W.host_pool_tensor(n_pool, 91, device=DEV)      # the follower's bf16 rows
    f_pool = torch.zeros((n_pool, 656), dtype=torch.uint8, pin_memory=True)
    hs.hs_quant_rows(layer.to(DEV), f_pool)
    f_hot = torch.zeros((n_hot, 656), dtype=torch.uint8, device=DEV)
    step = W.bf16_normal((cfg.B, cfg.d + 1, 576), 1.0, 5, "f-step").to(DEV)
    at = np.array([[b * S_tot + cfg.S + k for k in range(cfg.d + 1)] for b in range(cfg.B)], np.int32)
    hs.hs_quant_rows(step.view(-1, 576), f_hot, dst_slots=_t(at.reshape(-1)))
    torch.cuda.synchronize()
    e_hot = np.zeros((n_hot, 656), np.uint8)
    e_hot[at.reshape(-1)] = O.q8_quantise(_f64(step).reshape(-1, 576))
    e_pool = O.q8_quantise(_f64(layer))
    assert np.array_equal(f_pool.numpy(), e_pool)
    topk = W.topk_independent(cfg, 0, cfg.L, req, ri)
    wave = np.where(ri == 0)[0]
    clen = W.causal_lengths(cfg.L, req, ri)[wave]
    slot = torch.empty((len(wave), cfg.K), dtype=torch.int32, device=DEV)
    hs.hs_swap_in(buf, _t(req[wave]), _t(clen), hb["kv_len"], _t(topk[wave]), slot)
    e_slot, _, _, _ = ref.swap_in(req[wave], clen, cfg.L, topk[wave])
    hs.hs_swap_apply_plan(buf, [f_hot], [f_pool])
    O.apply_plan(ref.last_plan, e_hot, e_pool, hb["hbt_np"], cfg.block_size, S_tot)
    q = torch.as_tensor(np.random.default_rng(3).standard_normal((len(wave), cfg.H, 576)).astype(np.float32)).to(torch.bfloat16)
    out, lse = _attend(hs, q.to(DEV), f_hot, slot, cfg.scale, torch.empty(32 << 20, dtype=torch.uint8, device=DEV))
    assert np.array_equal(np_(slot), e_slot) and np.array_equal(np_(f_hot), e_hot)
    _check(out, lse, _f64(q), O.q8_values(e_hot), e_slot, cfg.scale)
    # sampled verify, commit
    g = np.random.default_rng(8)
    B, d, V = cfg.B, cfg.d, 300
    logits = torch.as_tensor((g.standard_normal((B, d + 1, V)) * 2).astype(np.float32))
    drafts = logits[:, :d].argmax(-1).int()
    u, E = g.random((B, d)).astype(np.float32) * 0.2, g.exponential(size=(B, V)).astype(np.float32)
    T = np.array([0.7] * B, np.float32)
    kv_len, skv = hb["kv_len"], W.step_kv(cfg, 0, device=DEV)
    acc = torch.empty(B, dtype=torch.int32, device=DEV)
    nxt, lp = torch.empty_like(acc), torch.empty((B, d + 1), device=DEV)
    hs.hs_verify_sample_finalize(buf, logits.to(DEV), _t(T), drafts.to(DEV), None, _t(u), _t(E), skv, kv_len,
                                 acc, nxt, logprob=lp)
    e_acc, e_nxt, e_lp, margin = O.verify_sample(logits, T, drafts, None, u, E)
    assert (margin > 1e-5).all()
    assert np.array_equal(np_(acc), e_acc) and np.array_equal(np_(nxt), e_nxt)
    ref.now += 1
    bits = skv.view(torch.int16).cpu().numpy().view(np.uint16)
    for b in range(B):
        assert ref.commit(b, int(cfg.L[b]), bits[b, :e_acc[b] + 1], ref.now)
    assert np.array_equal(np_(kv_len), np.asarray(cfg.L) + e_acc + 1)
    ts, stok, sts = buf.dump()
    for b in range(B):
        assert np.array_equal(ts[b].numpy(), ref.token_slot_array(b))
    assert hs.hs_get_status(buf) == 0
    buf.close()


def test_row_calls_from_and_to_host_memory_in_a_graph():
    """Pinned source rows into a device cache and its rows into pinned memory,
    captured once, replayed over new rows."""
    hs = lib()
    g = np.random.default_rng(13)
    n = 90
    src = _rows(g, n, torch.float32).pin_memory()
    cache = torch.zeros((n, 656), dtype=torch.uint8, device=DEV)
    back = torch.zeros((n, 576), dtype=torch.bfloat16).pin_memory()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        hs.hs_quant_rows(src, cache, status=st)
        hs.hs_dequant_rows(cache, back, status=st)
    for _ in range(2):
        src.copy_(_rows(g, n, torch.float32))
        gr.replay()
        torch.cuda.synchronize()
        want = O.q8_quantise(_f64(src))
        _check_bytes(np_(cache), want)
        assert np.array_equal(_f64(back), O.q8_values(want))
    assert int(st.item()) == 0


def test_row_calls_on_a_side_stream():
    hs = lib()
    g = np.random.default_rng(14)
    src = _rows(g, 3000, torch.bfloat16).to(DEV)
    cache = torch.zeros((3000, 656), dtype=torch.uint8, device=DEV)
    back = torch.zeros((3000, 576), dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    hs.hs_quant_rows(src, cache, stream=s)
    hs.hs_dequant_rows(cache, back, stream=s.cuda_stream)
    s.synchronize()
    assert np.array_equal(_f64(back), O.q8_values(O.q8_quantise(_f64(src))))


@pytest.mark.parametrize("H", [24, 9])
def test_attention_degenerate_calls_and_refusals(H):
    hs = lib()
    g = np.random.default_rng(15)
    rows, values = _cache(g, 300)
    cache = _t(rows)
    q = torch.as_tensor(g.standard_normal((2, H, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    idx = _t(_indices(g, 2, 700, 300, 0.1))
    ref, ref_lse = _attend(hs, q, cache, idx, 1 / 24)
    _check(ref, ref_lse, _f64(q), values, np_(idx), 1 / 24)
    # a workspace too small for two parts: one part, the same bits
    out, lse = _attend(hs, q, cache, idx, 1 / 24, torch.empty(160, dtype=torch.uint8, device=DEV))
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    # no lse wanted, whole and in parts
    big = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)
    whole, _ = _attend(hs, q, cache, idx, 1 / 24, big)
    for ws, want in ((None, ref), (big, whole)):
        out = torch.empty_like(ref)
        hs.hs_sparse_attn_decode_q8(q, cache, idx, 1 / 24, out, workspace=ws)
        assert torch.equal(out, want)
    # scale 0: the mean of the values, lse = ln of their number
    out, lse = _attend(hs, q, cache, idx, 0.0, big)
    _check(out, lse, _f64(q), values, np_(idx), 0.0)
    # no keys, an empty cache, no rows
    for c, i in ((cache, idx[:, :0].contiguous()), (cache[:0], idx)):
        out, lse = _attend(hs, q, c, i, 1 / 24, big)
        assert not out.any() and torch.isneginf(lse).all()
    hs.hs_sparse_attn_decode_q8(q[:0], cache, idx[:0], 1 / 24, ref[:0])
    for bad in (-0.1, float("inf"), float("nan")):
        with pytest.raises(hs.HisparseError):
            hs.hs_sparse_attn_decode_q8(q, cache, idx, bad, ref)
    with pytest.raises(hs.HisparseError):
        hs.hs_sparse_attn_decode_q8(q, cache, idx, 1 / 24, ref, workspace=big[8:])
    with pytest.raises(ValueError):
        hs.hs_sparse_attn_decode_q8(q, cache, idx[:1], 1 / 24, ref)
    with pytest.raises(ValueError):
        hs.hs_sparse_attn_decode_q8(q, cache[:, :655], idx, 1 / 24, ref)
    with pytest.raises(ValueError):
        hs.hs_sparse_attn_decode_q8(q, cache.cpu(), idx, 1 / 24, ref)
    with pytest.raises(TypeError):
        hs.hs_sparse_attn_decode_q8(q.float(), cache, idx, 1 / 24, ref)


@pytest.mark.parametrize("H", [50, 12])
def test_attention_leaves_its_neighbours_alone(H):
    """Outputs and workspace in the middle of larger buffers: nothing around
    them is written."""
    hs = lib()
    g = np.random.default_rng(16)
    rows, _ = _cache(g, 500)
    R, K = 3, 640
    q = torch.as_tensor(g.standard_normal((R, H, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    idx = _t(_indices(g, R, K, 500, 0.0))
    pad_o = torch.full((R * H * 512 + 256,), 3.0, dtype=torch.bfloat16, device=DEV)
    pad_l = torch.full((R * H + 32,), 3.0, device=DEV)
    parts = 5 if H > 16 else 10                            # 20 tiles of 32 keys, four or two to a part
    size = parts * R * H * 513 * 4
    pad_w = torch.full((size + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    out, lse = pad_o[128:128 + R * H * 512].view(R, H, 512), pad_l[16:16 + R * H].view(R, H)
    hs.hs_sparse_attn_decode_q8(q, _t(rows), idx, 1 / 24, out, lse=lse, workspace=pad_w[256:256 + size])
    want, want_lse = _attend(hs, q, _t(rows), idx, 1 / 24, torch.empty(32 << 20, dtype=torch.uint8, device=DEV))
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert (pad_o[:128] == 3).all() and (pad_o[-128:] == 3).all()
    assert (pad_l[:16] == 3).all() and (pad_l[-16:] == 3).all()
    assert (pad_w[:256] == 0x5A).all() and (pad_w[-256:] == 0x5A).all()


FIRST_CALLS = """
import torch
import hisparse_top_sparse_gb300 as hs
d = "cuda"
src = torch.randn((64, 576), device=d).bfloat16()
cache = torch.zeros((64, 656), dtype=torch.uint8, device=d)
back = torch.zeros((64, 576), dtype=torch.bfloat16, device=d)
q = torch.randn((2, 128, 576), device=d).bfloat16()
idx = torch.randint(0, 64, (2, 600), dtype=torch.int32, device=d)
ws = torch.empty(hs.ATTN_Q8_WORKSPACE_BYTES, dtype=torch.uint8, device=d)
outs = [torch.zeros((2, 128, 512), dtype=torch.bfloat16, device=d) for _ in range(2)]
v = (torch.randn((2, 3, 1000), device=d), torch.ones(2, device=d), torch.zeros((2, 2), dtype=torch.int32, device=d),
     None, torch.zeros((2, 2), device=d), torch.rand((2, 1000), device=d) + 0.1)
toks = [torch.full((2, 2), -7, dtype=torch.int32, device=d) for _ in range(2)]


def run(out, tok):
    hs.hs_quant_rows(src, cache)
    hs.hs_dequant_rows(cache, back)
    hs.hs_sparse_attn_decode_q8(q, cache, idx, 0.04, out, workspace=ws)
    hs.hs_verify_sample(*v, tok[0], tok[1])


torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run(outs[0], toks[0])
g.replay()
run(outs[1], toks[1])
torch.cuda.synchronize()
assert torch.equal(outs[0], outs[1]) and outs[0].abs().sum() > 0
assert torch.equal(toks[0], toks[1]) and (toks[0] >= 0).all()
"""


def test_the_first_calls_of_a_process_may_be_captured():
    lib()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
