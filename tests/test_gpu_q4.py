"""GPU parity of the 4-bit latent rows (hs_quant_rows_q4, hs_dequant_rows_q4) and
of the attention over them (hs_sparse_attn_decode_q4): bytes and values
bit-exact against the oracle, attention within bounds derived from its
roundings, and bit-identical to hs_sparse_attn_decode over the same values."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import hs_oracle as O
from gpu_util import lib, np_

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROW = 416


def _t(a):
    return torch.as_tensor(np.ascontiguousarray(a), device=DEV)


def _rows(g, n, dtype, width=576):
    x = g.standard_normal((n, width)) * np.exp(g.standard_normal((n, width)) * 2)
    return torch.as_tensor(x.astype(np.float32)).to(dtype)


def _f64(x):
    return x.detach().cpu().double().numpy()


def _check_bytes(got, want):
    """The codes of a group that is not finite say nothing."""
    assert np.array_equal(got[:, 384:], want[:, 384:])
    fine = np.repeat(want[:, 384:] != 255, 8, axis=1)
    assert np.array_equal(got[:, :256][fine], want[:, :256][fine])
    r = O.bf16_bits_to_f64(np.ascontiguousarray(want[:, 256:384]).view(np.uint16))
    s = O.bf16_bits_to_f64(np.ascontiguousarray(got[:, 256:384]).view(np.uint16))
    assert np.array_equal(r, s, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,width,offset", [(1, 576, 0), (7, 640, 64), (300, 1152, 8), (2500, 584, 8), (6001, 576, 0)])
def test_quant_rows_bytes(dtype, n, width, offset):
    hs = lib()
    g = np.random.default_rng(n + width)
    wide = _rows(g, n, dtype, width).to(DEV)
    src = wide[:, offset:offset + 576]
    rows = n + 11
    cache = torch.full((rows, ROW), 0xA5, dtype=torch.uint8, device=DEV)
    slots = g.permutation(rows)[:n].astype(np.int32)
    slots[::5] = -1
    hs.hs_quant_rows_q4(src, cache, dst_slots=_t(slots))
    want = np.full((rows, ROW), 0xA5, np.uint8)
    keep = slots >= 0
    if keep.any():
        want[slots[keep]] = O.q4_quantise(_f64(src)[keep])
    got = np_(cache)
    held = np.zeros(rows, bool)
    held[slots[keep]] = True
    assert np.array_equal(got[~held], want[~held])     # rows without an entry stay as they were
    if keep.any():
        _check_bytes(got[held], want[held])
    for out_t in (torch.float32, torch.bfloat16):
        back = torch.full((n, 640), 5.0, dtype=out_t, device=DEV)
        hs.hs_dequant_rows_q4(cache, back[:, 64:], src_slots=_t(slots))
        e = np.full((n, 640), 5.0)
        if keep.any():
            e[keep, 64:] = O.q4_values(want[slots[keep]])
        assert np.array_equal(_f64(back), e)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_rows_on_borders(dtype):
    """Numbers on the middles between two codes and next to them, and groups whose
    largest magnitude is six times a scale or next to that, for all scales."""
    hs = lib()
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x = np.zeros((255, 32, 16), np.float32)
    for b in range(255):
        s = np.float32(O.Q4_SCALES[b])
        for k in range(24):                            # the middles, and a step up and down (f32)
            v = (mids * float(s)).astype(np.float32)
            v = v if k % 3 == 0 else np.nextafter(v, np.float32(np.inf if k % 3 == 1 else 0))
            x[b, k, :8], x[b, k, 8:] = v, -v[::-1]
            if k % 3 == 1 and k < 12:
                x[b, k, 7], x[b, k, 8] = 0, 0          # without it the group's scale is the next one
        for k in range(24, 32):
            x[b, k, k - 24] = [6 * s, np.nextafter(6 * s, np.float32(0)), np.nextafter(6 * s, np.float32(np.inf)), s,
                               6 * s * np.float32(1.03), s * np.float32(0.1), 6 * s, -6 * s][k - 24]
    src = torch.zeros((255, 576), dtype=torch.float32)
    src[:, :512] = torch.from_numpy(x.reshape(255, 512))
    src = src.to(dtype)
    cache = torch.empty((255, ROW), dtype=torch.uint8, device=DEV)
    hs.hs_quant_rows_q4(src.to(DEV), cache)
    _check_bytes(np_(cache), O.q4_quantise(_f64(src)))


def test_quant_rows_special_values():
    hs = lib()
    x = torch.zeros((6, 576))
    x[0, ::16] = torch.tensor([0.0, 6, 6.001, 1e-38, 1e-45, 2.0 ** -17, 2.0 ** -18, 344064, 344065, 2.0 ** 127, 3.0e38,
                               3.4e38, -6, 5.0001, -0.0, 5, 6, 7] * 2)[:36]
    x[1, 0], x[1, 1] = float("nan"), 3.0
    x[1, 32], x[1, 33], x[1, 64] = float("inf"), 1.0, -float("inf")
    x[1, 100] = -float("nan")
    x[1, 575], x[1, 574] = float("nan"), float("inf")
    x[2, :512] = torch.linspace(-6, 6, 512)
    x[3, :512] = float(torch.finfo(torch.float32).max)
    x[4, :512] = 2.0 ** torch.arange(-256, 256).float().clamp(-149, 127)
    x[5, :512] = float("nan")
    for dtype in (torch.float32, torch.bfloat16):
        src = x.to(dtype)
        cache = torch.empty((6, ROW), dtype=torch.uint8, device=DEV)
        hs.hs_quant_rows_q4(src.to(DEV), cache)
        want = O.q4_quantise(_f64(src))
        _check_bytes(np_(cache), want)
        for out_t in (torch.float32, torch.bfloat16):
            back = torch.empty((6, 576), dtype=out_t, device=DEV)
            hs.hs_dequant_rows_q4(cache, back)
            assert np.array_equal(_f64(back), O.q4_values(want), equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequant_rows_every_code_and_scale(dtype):
    hs = lib()
    g = np.random.default_rng(4)
    rows = np.zeros((300, ROW), np.uint8)
    rows[:, :256] = (np.arange(256) + np.arange(300)[:, None] * 7) % 256
    rows[:, 256:384] = g.integers(0, 127, (300, 128))       # finite bf16 values
    rows[:256, 384:] = np.arange(256)[:, None]              # (255: NaN)
    rows[256:, 384:] = g.integers(0, 256, (44, 32))
    rows[299] = 0                                           # a row never written
    want = O.q4_values(rows)
    slots = g.integers(-1, 300, size=1000).astype(np.int32)
    slots[:300] = np.arange(300)
    dst = g.permutation(1100)[:1000].astype(np.int32)
    dst[3::50] = -1
    wide = torch.full((1100, 640), 7.0, dtype=dtype, device=DEV)
    hs.hs_dequant_rows_q4(_t(rows), wide[:, 64:], src_slots=_t(slots), dst_slots=_t(dst))
    e = np.full((1100, 640), 7.0)
    keep = (slots >= 0) & (dst >= 0)
    e[dst[keep], 64:] = want[slots[keep]]
    assert np.array_equal(_f64(wide), e, equal_nan=True)


def test_row_calls_report_bad_slots_and_leave_the_rest():
    hs = lib()
    g = np.random.default_rng(5)
    src = _rows(g, 10, torch.bfloat16).to(DEV)
    cache = torch.zeros((12, ROW), dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    s = np.array([0, 10, 3, -1, 5], np.int32)
    d = np.array([2, 3, 12, 4, 5], np.int32)
    hs.hs_quant_rows_q4(src, cache, src_slots=_t(s), dst_slots=_t(d), status=st)
    assert int(st.item()) == hs.HS_STATUS_INDEX
    want = np.zeros((12, ROW), np.uint8)
    want[[2, 5]] = O.q4_quantise(_f64(src)[[0, 5]])
    assert np.array_equal(np_(cache), want)
    st.zero_()
    back = torch.full((4, 576), 9.0, device=DEV)
    hs.hs_dequant_rows_q4(cache, back, src_slots=_t(np.array([2, 12, 5], np.int32)),
                          dst_slots=_t(np.array([1, 0, 4], np.int32)), status=st)
    assert int(st.item()) == hs.HS_STATUS_INDEX
    e = np.full((4, 576), 9.0)
    e[1] = O.q4_values(want[2:3])[0]
    assert np.array_equal(_f64(back), e)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    hs.hs_quant_rows_q4(src, cache, src_slots=none, dst_slots=none)
    with pytest.raises(ValueError):
        hs.hs_quant_rows_q4(src, cache[:4])                   # ten rows into four
    with pytest.raises(ValueError):
        hs.hs_quant_rows_q4(src, cache, src_slots=_t(s), dst_slots=_t(d[:3]))
    with pytest.raises(ValueError):
        hs.hs_quant_rows_q4(src.t().contiguous().t(), cache)
    with pytest.raises(ValueError):
        hs.hs_quant_rows_q4(src, torch.zeros((12, 656), dtype=torch.uint8, device=DEV))
    with pytest.raises(hs.HisparseError):
        hs.hs_quant_rows_q4(torch.zeros((4, 577), dtype=torch.bfloat16, device=DEV)[:, 1:], cache)


def test_row_calls_from_and_to_host_memory_on_streams_and_in_a_graph():
    hs = lib()
    g = np.random.default_rng(13)
    n = 90
    src = _rows(g, n, torch.float32).pin_memory()
    cache = torch.zeros((n, ROW), dtype=torch.uint8).pin_memory()
    back = torch.zeros((n, 576), dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    hs.hs_quant_rows_q4(src, cache, status=st, stream=side)
    hs.hs_dequant_rows_q4(cache, back, status=st, stream=side.cuda_stream)
    side.synchronize()
    want = O.q4_quantise(_f64(src))
    _check_bytes(cache.numpy(), want)
    assert np.array_equal(_f64(back), O.q4_values(want))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        hs.hs_quant_rows_q4(src, cache, status=st)
        hs.hs_dequant_rows_q4(cache, back, status=st)
    for _ in range(2):
        src.copy_(_rows(g, n, torch.float32))
        gr.replay()
        torch.cuda.synchronize()
        want = O.q4_quantise(_f64(src))
        _check_bytes(cache.numpy(), want)
        assert np.array_equal(_f64(back), O.q4_values(want))
    assert int(st.item()) == 0


# ------------------------------------------------------------- attention --

def _cache(g, n):
    """q4 rows of latent-like values, and their values."""
    rows = O.q4_quantise(g.standard_normal((n, 576)) * np.exp(0.5 * g.standard_normal((1, 576))))
    return rows, O.q4_values(rows)


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
    hs.hs_sparse_attn_decode_q4(q, cache, idx, scale, out, lse=lse, workspace=ws, status=st, **kw)
    assert int(st.item()) == 0
    return out, lse


def _q(g, R, H):
    return torch.as_tensor(g.standard_normal((R, H, 576)).astype(np.float32)).to(torch.bfloat16)


def _space(size=32 << 20):
    return torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)


CASES = [(1, 1, 1, 0.0), (3, 16, 5, 0.0), (2, 128, 2048, 0.0), (5, 40, 33, 0.3), (2, 136, 130, 0.1),
         (1, 128, 8192, 0.05), (80, 128, 96, 0.5), (9, 64, 1000, 0.9), (1, 1024, 300, 0.0), (3, 128, 32, 0.0),
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
    q = _q(g, R, H)
    scale = 1 / 24
    ws = _space(workspace) if workspace else None
    out, lse = _attend(hs, q.to(DEV), _t(rows), _t(idx), scale, ws)
    _check(out, lse, _f64(q), values, idx, scale)
    again, lse2 = _attend(hs, q.to(DEV), _t(rows), _t(idx), scale, ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("R,H,K", [(3, 128, 2048), (100, 128, 200), (2, 20, 77)])
def test_attention_equals_the_bf16_call_over_the_same_values(R, H, K):
    """Without a workspace the tiles, their order and their values (2^-15 of
    them) are those of hs_sparse_attn_decode over the rows read back."""
    hs = lib()
    g = np.random.default_rng(R + K)
    rows, values = _cache(g, 3000)
    idx = _t(_indices(g, R, K, 3000, 0.1))
    q = _q(g, R, H).to(DEV)
    cache = _t(rows)
    wide = torch.empty((3000, 576), dtype=torch.bfloat16, device=DEV)
    hs.hs_dequant_rows_q4(cache, wide)
    out, lse = _attend(hs, q, cache, idx, 0.04)
    ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
    hs.hs_sparse_attn_decode(q, wide, idx, 0.04, ref, lse=ref_lse)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("H", [128, 16])
def test_attention_over_every_scale(H):
    """Rows whose values fill the format's range, from 2^-17 to 6 * 2^15."""
    hs = lib()
    g = np.random.default_rng(21)
    x = g.standard_normal((255, 576)) * 1e-3
    x[:, :512] = g.standard_normal((255, 512)).clip(-3, 3) * np.repeat(O.Q4_SCALES[:, None], 512, 1)
    rows = O.q4_quantise(x)
    values = O.q4_values(rows)
    idx = np.stack([np.arange(255), np.arange(255)[::-1]]).astype(np.int32)
    q = _q(g, 2, H)
    scale = 1e-6
    for ws in (None, _space()):
        out, lse = _attend(hs, q.to(DEV), _t(rows), _t(idx), scale, ws)
        _check(out, lse, _f64(q), values, idx, scale)


@pytest.mark.parametrize("H", [128, 16])
def test_attention_second_pass_and_sharp_logits(H):
    """Scores whose later tiles pass the first ones by more than 2^30."""
    hs = lib()
    g = np.random.default_rng(9)
    x = g.standard_normal((600, 576))
    x[300:] *= 40
    rows = O.q4_quantise(x)
    values = O.q4_values(rows)
    idx = np.arange(600, dtype=np.int32)[None].repeat(3, 0)
    q = _q(g, 3, H)
    for ws in (None, _space()):
        out, lse = _attend(hs, q.to(DEV), _t(rows), _t(idx), 0.25, ws)
        _check(out, lse, _f64(q), values, idx, 0.25)


@pytest.mark.parametrize("H", [8, 40])
def test_attention_ignores_what_it_does_not_select(H):
    """NaN and infinity in rows that no index names, exact single keys, and
    duplicates counted each time."""
    hs = lib()
    g = np.random.default_rng(10)
    rows, values = _cache(g, 64)
    rows[40:, 384:] = 255
    rows[40:, 256:384] = 0xFF
    q = _q(g, 2, H)
    idx = np.array([[-1, 7, -1, 64], [3, 3, 5, -7]], np.int32)
    out, lse = _attend(hs, q.to(DEV), _t(rows), _t(idx), 1 / 24)
    _check(out, lse, _f64(q), values, idx, 1 / 24)
    assert torch.equal(out[0].cpu(), torch.as_tensor(values[7, :512]).to(torch.bfloat16).expand(H, 512))
    # a selected NaN row reaches the output in every split
    idx = np.zeros((1, 2048), np.int32)
    idx[0, 2000] = 50
    for ws in (None, _space()):
        out, lse = _attend(hs, q[:1].to(DEV), _t(rows), _t(idx), 1 / 24, ws)
        assert out.isnan().all()


def test_attention_in_a_cache_past_4_gib():
    """Row offsets past 32 bits."""
    hs = lib()
    g = np.random.default_rng(11)
    n = (1 << 32) // ROW + 1000
    rows, values = _cache(g, 512)
    cache = torch.zeros((n, ROW), dtype=torch.uint8, device=DEV)
    at = np.sort(g.permutation(900)[:512]) + n - 900
    hs.hs_quant_rows_q4(_t(values.astype(np.float32)), cache, dst_slots=_t(at.astype(np.int32)))
    idx = at[g.integers(0, 512, size=(2, 600))].astype(np.int32)
    for H in (128, 7):
        q = _q(g, 2, H)
        out, lse = _attend(hs, q.to(DEV), cache, _t(idx), 1 / 24, _space())
        _check(out, lse, _f64(q), values, np.searchsorted(at, idx).astype(np.int32), 1 / 24)
    back = torch.empty((3, 576), device=DEV)
    hs.hs_dequant_rows_q4(cache, back, src_slots=_t(at[-3:].astype(np.int32)))
    assert np.array_equal(_f64(back), values[-3:])


@pytest.mark.parametrize("H", [128, 10])
def test_attention_on_a_side_stream_and_in_graphs(H):
    """Two captured calls, a workspace each, replayed on two streams at once
    over new inputs; the eager call on a side stream."""
    hs = lib()
    g = np.random.default_rng(12)
    rows, _ = _cache(g, 900)
    cache = _t(rows)
    mk = lambda: (_q(g, 3, H).to(DEV), _t(_indices(g, 3, 1500, 900, 0.1)))
    ins = [mk(), mk()]
    ws = [_space() for _ in range(2)]
    outs = [_attend(hs, q, cache, idx, 1 / 24, w) for (q, idx), w in zip(ins, ws)]
    got = [(torch.empty_like(o), torch.empty_like(l)) for o, l in outs]
    graphs = []
    for i, (q, idx) in enumerate(ins):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            hs.hs_sparse_attn_decode_q4(q, cache, idx, 1 / 24, got[i][0], lse=got[i][1], workspace=ws[i])
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


@pytest.mark.parametrize("H", [24, 9])
def test_attention_degenerate_calls_and_refusals(H):
    hs = lib()
    g = np.random.default_rng(15)
    rows, values = _cache(g, 300)
    cache = _t(rows)
    q = _q(g, 2, H).to(DEV)
    idx = _t(_indices(g, 2, 700, 300, 0.1))
    ref, ref_lse = _attend(hs, q, cache, idx, 1 / 24)
    _check(ref, ref_lse, _f64(q), values, np_(idx), 1 / 24)
    # a workspace too small for two parts: one part, the same bits
    out, lse = _attend(hs, q, cache, idx, 1 / 24, _space(160))
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    # no lse wanted, whole and in parts
    big = _space()
    whole, _ = _attend(hs, q, cache, idx, 1 / 24, big)
    for ws, want in ((None, ref), (big, whole)):
        out = torch.empty_like(ref)
        hs.hs_sparse_attn_decode_q4(q, cache, idx, 1 / 24, out, workspace=ws)
        assert torch.equal(out, want)
    # scale 0: the mean of the values, lse = ln of their number
    out, lse = _attend(hs, q, cache, idx, 0.0, big)
    _check(out, lse, _f64(q), values, np_(idx), 0.0)
    # no keys, an empty cache, no rows
    for c, i in ((cache, idx[:, :0].contiguous()), (cache[:0], idx)):
        out, lse = _attend(hs, q, c, i, 1 / 24, big)
        assert not out.any() and torch.isneginf(lse).all()
    hs.hs_sparse_attn_decode_q4(q[:0], cache, idx[:0], 1 / 24, ref[:0])
    for bad in (-0.1, 2.0 ** 101, float("inf"), float("nan")):
        with pytest.raises(hs.HisparseError):
            hs.hs_sparse_attn_decode_q4(q, cache, idx, bad, ref)
    with pytest.raises(hs.HisparseError):
        hs.hs_sparse_attn_decode_q4(q, cache, idx, 1 / 24, ref, workspace=big[8:])
    with pytest.raises(ValueError):
        hs.hs_sparse_attn_decode_q4(q, cache, idx[:1], 1 / 24, ref)
    with pytest.raises(ValueError):
        hs.hs_sparse_attn_decode_q4(q, torch.zeros((300, 656), dtype=torch.uint8, device=DEV), idx, 1 / 24, ref)
    with pytest.raises(ValueError):
        hs.hs_sparse_attn_decode_q4(q, cache.cpu(), idx, 1 / 24, ref)
    with pytest.raises(TypeError):
        hs.hs_sparse_attn_decode_q4(q.float(), cache, idx, 1 / 24, ref)


@pytest.mark.parametrize("H", [50, 12])
def test_attention_leaves_its_neighbours_alone(H):
    """Outputs and workspace in the middle of larger buffers: nothing around
    them is written."""
    hs = lib()
    g = np.random.default_rng(16)
    rows, _ = _cache(g, 500)
    R, K = 3, 640
    q = _q(g, R, H).to(DEV)
    idx = _t(_indices(g, R, K, 500, 0.0))
    pad_o = torch.full((R * H * 512 + 256,), 3.0, dtype=torch.bfloat16, device=DEV)
    pad_l = torch.full((R * H + 32,), 3.0, device=DEV)
    pad_w = _space()
    out, lse = pad_o[128:128 + R * H * 512].view(R, H, 512), pad_l[16:16 + R * H].view(R, H)
    parts = 10                                             # 20 tiles of 32 keys, two or more to a part
    size = parts * R * H * 513 * 4
    hs.hs_sparse_attn_decode_q4(q, _t(rows), idx, 1 / 24, out, lse=lse, workspace=pad_w[256:256 + size])
    want, want_lse = _attend(hs, q, _t(rows), idx, 1 / 24, _space())
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert (pad_o[:128] == 3).all() and (pad_o[-128:] == 3).all()
    assert (pad_l[:16] == 3).all() and (pad_l[-16:] == 3).all()
    assert (pad_w[:256] == 0xFF).all() and (pad_w[256 + size:] == 0xFF).all()


def test_a_step_over_a_q4_follower_layer_with_rotated_rows():
    """The operators as a step uses them: latent rows rotated by their positions,
    quantised into a follower's host pool and step slots, the leader's swap-in,
    its plan repeated for the 416-byte rows, q rotated in place, attention over
    the follower through the leader's slot table; once eagerly and once more
    (rotation, quantising, attention) from a graph."""
    hs = lib()
    cfg = W.get_config(1)
    req, ri = W.rows_of(cfg)
    hb = W.host_backed_case(cfg, device=DEV, extra_positions=8)
    buf = hs.HsBuffer(cfg.B, cfg.S, cfg.d + 1, hb["max_ctx"], cfg.block_size, hb["hot"], hb["pool"], hb["hbt"])
    ref = O.HotBuffer(cfg.B, cfg.S, cfg.d + 1, hb["max_ctx"], cfg.block_size, hb["hbt_np"], hb["pool"].clone())
    n_pool, n_hot, S_tot = hb["pool"].shape[0], hb["hot"].shape[0], cfg.S + cfg.d + 1
    freqs, factor = hs.hs_rope_freqs(64, scaling=hs.HS_ROPE_YARN, scale=40.0, context=4096)
    d_freqs = freqs.to(DEV)
    # the follower's rows, each rotated by the position its host row belongs to
    layer = W.host_pool_tensor(n_pool, 91, device=DEV).to(DEV)
    pos = np.zeros(n_pool, np.int32)
    for b in range(cfg.B):
        for k in range(hb["hbt_np"].shape[1]):
            at = hb["hbt_np"][b, k] * cfg.block_size
            if 0 <= at < n_pool:                            # (blocks past a request's length are none)
                pos[at:at + cfg.block_size] = np.arange(k * cfg.block_size, (k + 1) * cfg.block_size)
    rot = layer.clone()
    hs.hs_rope_rows(rot, rot, _t(pos), d_freqs, factor=factor, rot_off=512)
    f_pool = torch.zeros((n_pool, ROW), dtype=torch.uint8, pin_memory=True)
    hs.hs_quant_rows_q4(rot, f_pool)
    f_hot = torch.zeros((n_hot, ROW), dtype=torch.uint8, device=DEV)
    step = W.bf16_normal((cfg.B * (cfg.d + 1), 576), 1.0, 5, "f-step").to(DEV)
    step_pos = np.array([cfg.L[b] + k for b in range(cfg.B) for k in range(cfg.d + 1)], np.int32)
    at = np.array([b * S_tot + cfg.S + k for b in range(cfg.B) for k in range(cfg.d + 1)], np.int32)
    turned = torch.empty_like(step)

    def write_step():
        hs.hs_rope_rows(step, turned, _t_pos, d_freqs, factor=factor, rot_off=512)
        hs.hs_quant_rows_q4(turned, f_hot, dst_slots=_t_at)

    _t_pos, _t_at = _t(step_pos), _t(at)
    write_step()
    torch.cuda.synchronize()
    want = O.rope_rows(_f64(layer)[:, None], pos, freqs.numpy(), factor, 512)[:, 0]
    assert np.array_equal(_f64(rot)[:, :512], _f64(layer)[:, :512])
    assert (np.abs(_f64(rot) - want) <= np.abs(want) * 2.0 ** -8 + 2.0 ** -19 * factor * np.abs(_f64(layer)).max()).all()
    e_pool = O.q4_quantise(_f64(rot))
    _check_bytes(f_pool.numpy(), e_pool)
    e_hot = np.zeros((n_hot, ROW), np.uint8)
    e_hot[at] = O.q4_quantise(_f64(turned))
    topk = W.topk_independent(cfg, 0, cfg.L, req, ri)
    wave = np.where(ri == 0)[0]
    clen = W.causal_lengths(cfg.L, req, ri)[wave]
    slot = torch.empty((len(wave), cfg.K), dtype=torch.int32, device=DEV)
    hs.hs_swap_in(buf, _t(req[wave]), _t(clen), hb["kv_len"], _t(topk[wave]), slot)
    e_slot, _, _, _ = ref.swap_in(req[wave], clen, cfg.L, topk[wave])
    hs.hs_swap_apply_plan(buf, [f_hot], [f_pool])
    O.apply_plan(ref.last_plan, e_hot, e_pool, hb["hbt_np"], cfg.block_size, S_tot)
    raw = _q(np.random.default_rng(3), len(wave), cfg.H).to(DEV)
    q = raw.clone()
    q_pos = _t((clen - 1).astype(np.int32))
    hs.hs_rope_rows(q, q, q_pos, d_freqs, factor=factor, rot_off=512)
    ws = _space()
    out, lse = _attend(hs, q, f_hot, slot, cfg.scale, ws)
    assert np.array_equal(np_(slot), e_slot)
    _check_bytes(np_(f_hot), e_hot)
    _check(out, lse, _f64(q), O.q4_values(e_hot), e_slot, cfg.scale)
    got = torch.zeros_like(out)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        write_step()
        q.copy_(raw)
        hs.hs_rope_rows(q, q, q_pos, d_freqs, factor=factor, rot_off=512)
        hs.hs_sparse_attn_decode_q4(q, f_hot, slot, cfg.scale, got, workspace=ws)
    for _ in range(2):
        got.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    assert hs.hs_get_status(buf) == 0
    buf.close()
