"""GPU parity of the rotary positions (hs_rope_rows) with the oracle in 64 bits,
within bounds derived from the roundings."""
import numpy as np
import pytest
import torch

from oracle import hs_oracle as O
from gpu_util import lib, np_

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _t(a):
    return torch.as_tensor(np.ascontiguousarray(a), device=DEV)


def _f64(x):
    return x.detach().cpu().double().numpy()


def _bound(x, want, factor, dtype):
    """A cosine or sine is off by at most 2^-22 (its argument's roundings to f32,
    pi / 4 2^-23, a unit or two of 2^-24 for itself, and the factor's product), the
    two products and their sum by 2^-22 of the magnitudes more; then the rounding
    to the type, half a step."""
    a = np.abs(x).max(-1, keepdims=True)
    half = torch.finfo(dtype).eps / 2
    return 2 * a * abs(factor) * 2.0 ** -21 * (1 + half) + np.abs(want) * half + 1e-38


def _freqs(hs, rot, far):
    return hs.hs_rope_freqs(rot, scaling=hs.HS_ROPE_YARN if far else hs.HS_ROPE_PLAIN, scale=16.0, context=4096.0)


SHAPES = [  # rows, heads, dims, offset, rotated, wider source, wider destination
    (1, 1, 2, 0, 2, 0, 0), (5, 3, 64, 0, 64, 0, 0), (4, 128, 64, 0, 64, 128, 512), (33, 1, 576, 512, 64, 0, 64),
    (7, 5, 192, 0, 32, 0, 0), (9, 2, 128, 96, 32, 8, 24), (3, 40, 96, 8, 80, 0, 0), (2, 1, 256, 0, 256, 0, 0),
    (6, 7, 21, 3, 10, 0, 0), (5, 4, 66, 1, 64, 1, 3), (700, 16, 64, 0, 64, 0, 0), (3, 2, 4096, 1024, 2048, 0, 0),
    (11, 1, 24, 0, 24, 0, 0), (2000, 8, 128, 64, 64, 0, 0), (2, 301, 20, 4, 12, 0, 0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,H,dim,off,rot,more_src,more_dst", SHAPES)
def test_rows_against_the_oracle(n, H, dim, off, rot, more_src, more_dst, half, dtype):
    hs = lib()
    g = np.random.default_rng(n * 1009 + H * 31 + dim + half)
    src = torch.as_tensor(g.standard_normal((n, H, dim + more_src)).astype(np.float32)).to(dtype).to(DEV)[:, :, more_src:]
    wide = torch.full((n, H, dim + more_dst), 7.0, dtype=dtype, device=DEV)
    dst = wide[:, :, more_dst:]
    pos = g.integers(0, 1 << 20, size=n).astype(np.int32)
    pos[0] = 0
    freqs, factor = _freqs(hs, rot, n % 2)
    hs.hs_rope_rows(src, dst, _t(pos), freqs.to(DEV), factor=factor, rot_off=off,
                    layout=hs.HS_ROPE_HALF if half else hs.HS_ROPE_INTERLEAVED)
    x = _f64(src)
    want = O.rope_rows(x, pos, freqs.numpy(), factor, off, half)
    got = _f64(dst)
    assert (np.abs(got - want) <= _bound(x, want, factor, dtype)).all()
    beside = np.ones(dim, bool)
    beside[off:off + rot] = False
    assert np.array_equal(got[:, :, beside], x[:, :, beside])
    assert (wide[:, :, :more_dst] == 7).all()
    # in place: the same bits
    hs.hs_rope_rows(src, src, _t(pos), freqs.to(DEV), factor=factor, rot_off=off,
                    layout=hs.HS_ROPE_HALF if half else hs.HS_ROPE_INTERLEAVED)
    assert torch.equal(src, dst)


@pytest.mark.parametrize("half", [False, True])
def test_far_and_negative_positions(half):
    """Any position of 32 bits: the angle is exact modulo a turn."""
    hs = lib()
    g = np.random.default_rng(2)
    pos = np.array([2 ** 31 - 1, -2 ** 31, -1, 1, 10 ** 9, 123456789, -77777], np.int32)
    x = g.standard_normal((len(pos), 2, 64)).astype(np.float32)
    freqs, _ = hs.hs_rope_freqs(64)
    out = torch.empty((len(pos), 2, 64), device=DEV)
    hs.hs_rope_rows(_t(x), out, _t(pos), freqs.to(DEV), layout=int(half))
    want = O.rope_rows(x.astype(np.float64), pos, freqs.numpy(), 1.0, 0, half)
    assert (np.abs(_f64(out) - want) <= _bound(x, want, 1.0, torch.float32)).all()
    # any 64-bit fraction of a turn, negative ones and halves among them
    odd = np.array([-1, -(1 << 63), 1 << 62, (1 << 63) - 1, 12345678901234567], np.int64)
    y = x[:, :, :10].copy()
    hs.hs_rope_rows(_t(y), out[:, :, :10], _t(pos), _t(odd), layout=int(half))
    want = O.rope_rows(y.astype(np.float64), pos, odd, 1.0, 0, half)
    assert (np.abs(_f64(out[:, :, :10]) - want) <= _bound(y, want, 1.0, torch.float32)).all()


@pytest.mark.parametrize("half", [False, True])
def test_the_inverse_is_the_gradient(half):
    """Against the formula (the transposed rotation, times the factor), against
    differences of the forward call, which is linear, and with factor 1 as the
    way back."""
    hs = lib()
    g = np.random.default_rng(3)
    n, H, dim, off, rot, factor = 6, 3, 40, 4, 32, 1.25
    pos = _t(g.integers(0, 100000, size=n).astype(np.int32))
    freqs, _ = hs.hs_rope_freqs(rot)
    kw = dict(rot_off=off, layout=int(half))
    x, dy = (torch.as_tensor(g.standard_normal((n, H, dim)).astype(np.float32), device=DEV) for _ in range(2))
    d_freqs, dx = freqs.to(DEV), torch.empty((n, H, dim), device=DEV)
    hs.hs_rope_rows(dy, dx, pos, d_freqs, factor=factor, inverse=True, **kw)
    want = O.rope_rows(_f64(dy), np_(pos), freqs.numpy(), factor, off, half, inverse=True)
    assert (np.abs(_f64(dx) - want) <= _bound(_f64(dy), want, factor, torch.float32)).all()
    # d <dy, rope(x)> along a random direction v
    v = torch.as_tensor(g.standard_normal((n, H, dim)).astype(np.float32), device=DEV)
    up, down = torch.empty_like(x), torch.empty_like(x)
    hs.hs_rope_rows(x + v, up, pos, d_freqs, factor=factor, **kw)
    hs.hs_rope_rows(x - v, down, pos, d_freqs, factor=factor, **kw)
    diff = ((_f64(up) - _f64(down)) / 2 * _f64(dy)).sum()
    along = (_f64(dx) * _f64(v)).sum()
    # each of the values in the sums is off by some units of 2^-21 of the largest
    most = max(float(t.abs().max()) for t in (x + v, x - v, dy, v)) ** 2 * factor
    assert abs(diff - along) <= n * H * dim * most * 2.0 ** -19
    back = torch.empty_like(x)
    hs.hs_rope_rows(x, up, pos, d_freqs, **kw)
    hs.hs_rope_rows(up, back, pos, d_freqs, inverse=True, **kw)
    assert (np.abs(_f64(back) - _f64(x)) <= 2 * _bound(_f64(up), _f64(x), 1.0, torch.float32)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slots_status_and_rows_left_alone(dtype):
    hs = lib()
    g = np.random.default_rng(4)
    src = torch.as_tensor(g.standard_normal((10, 576)).astype(np.float32)).to(dtype).to(DEV)
    freqs, _ = hs.hs_rope_freqs(64)
    d_freqs = freqs.to(DEV)
    s = np.array([0, 10, 3, -1, 5, 7, 5], np.int32)
    d = np.array([2, 3, 12, 4, 5, -3, 0], np.int32)
    pos = g.integers(0, 9999, size=7).astype(np.int32)
    cache = torch.full((12, 576), 3.0, dtype=dtype, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    hs.hs_rope_rows(src, cache, _t(pos), d_freqs, rot_off=512, src_slots=_t(s), dst_slots=_t(d), status=st)
    assert int(st.item()) == hs.HS_STATUS_INDEX
    want = np.full((12, 576), 3.0)
    ok = [0, 4, 6]
    y = O.rope_rows(_f64(src)[s[ok]][:, None], pos[ok], freqs.numpy(), 1.0, 512)[:, 0]
    want[d[ok]] = y
    got = _f64(cache)
    written = np.isin(np.arange(12), d[ok])
    assert np.array_equal(got[~written], want[~written])
    b = _bound(_f64(src)[s[ok]], y, 1.0, dtype)
    assert (np.abs(got[d[ok]] - y) <= b).all()
    # cached rows moved to other positions where they lie
    st.zero_()
    slots = _t(np.array([5, 0], np.int32))
    before = _f64(cache)
    hs.hs_rope_rows(cache, cache, _t(np.array([100, -100], np.int32)), d_freqs, rot_off=512, src_slots=slots, dst_slots=slots,
                    status=st)
    y = O.rope_rows(before[[5, 0]][:, None], [100, -100], freqs.numpy(), 1.0, 512)[:, 0]
    got = _f64(cache)
    assert (np.abs(got[[5, 0]] - y) <= _bound(before[[5, 0]], y, 1.0, dtype)).all()
    rest = [r for r in range(12) if r not in (0, 5)]
    assert np.array_equal(got[rest], before[rest]) and int(st.item()) == 0
    # non-finite numbers go where they belong: rotated ones into their pair, others as they are
    src[0, 0], src[0, 512], src[1, 513] = float("nan"), float("inf"), float("nan")
    hs.hs_rope_rows(src[:2], cache[:2], _t(np.array([1, 1], np.int32)), d_freqs, rot_off=512)
    bad = ~torch.isfinite(cache[:2])
    assert bad[0, 0] and bad[0, 512] and bad[0, 513] and bad[1, 512] and bad[1, 513] and int(bad.sum()) == 5


def test_layouts_of_rows_and_heads():
    """Heads outside rows, a row shared by all sources, single rows of any stride."""
    hs = lib()
    g = np.random.default_rng(5)
    n, H = 9, 4
    pos = _t(g.integers(0, 5000, size=n).astype(np.int32))
    freqs, _ = hs.hs_rope_freqs(64)
    d_freqs = freqs.to(DEV)
    x = torch.as_tensor(g.standard_normal((H, n, 64)).astype(np.float32), device=DEV).transpose(0, 1)
    out = torch.zeros((H, n, 64), device=DEV)
    hs.hs_rope_rows(x, out.transpose(0, 1), pos, d_freqs)
    want = O.rope_rows(_f64(x), np_(pos), freqs.numpy())
    assert (np.abs(_f64(out.transpose(0, 1)) - want) <= _bound(_f64(x), want, 1.0, torch.float32)).all()
    one = x[:1].expand(n, H, 64)
    dst = torch.zeros((n, H, 64), device=DEV)
    hs.hs_rope_rows(one, dst, pos, d_freqs)
    want = O.rope_rows(_f64(one), np_(pos), freqs.numpy())
    assert (np.abs(_f64(dst) - want) <= _bound(_f64(one), want, 1.0, torch.float32)).all()
    hs.hs_rope_rows(x[:0], dst[:0], pos[:0], d_freqs)
    # no unaligned place is refused
    flat = torch.zeros(n * 64 + 1, dtype=torch.bfloat16, device=DEV)
    odd = flat[1:].view(n, 64)
    odd.copy_(x[:, 0])
    e = _f64(odd)
    hs.hs_rope_rows(odd, odd, pos, d_freqs)
    want = O.rope_rows(e[:, None], np_(pos), freqs.numpy())[:, 0]
    assert (np.abs(_f64(odd) - want) <= _bound(e, want, 1.0, torch.bfloat16)).all() and flat[0] == 0


def test_host_memory_streams_graphs():
    hs = lib()
    g = np.random.default_rng(6)
    n = 70
    freqs, _ = hs.hs_rope_freqs(64)
    d_freqs = freqs.to(DEV)
    pos = _t(g.integers(0, 5000, size=n).astype(np.int32))
    src = torch.as_tensor(g.standard_normal((n, 2, 96)).astype(np.float32)).pin_memory()
    dst = torch.zeros((n, 2, 96), device=DEV)
    back = torch.zeros((n, 2, 96)).pin_memory()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    hs.hs_rope_rows(src, dst, pos, d_freqs, rot_off=16, stream=side)
    hs.hs_rope_rows(dst, back, pos, d_freqs, rot_off=16, inverse=True, stream=side.cuda_stream)
    side.synchronize()
    want = O.rope_rows(_f64(src), np_(pos), freqs.numpy(), 1.0, 16)
    b = _bound(_f64(src), want, 1.0, torch.float32)
    assert (np.abs(_f64(dst) - want) <= b).all()
    assert (np.abs(_f64(back) - _f64(src)) <= 3 * b).all()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        hs.hs_rope_rows(src, dst, pos, d_freqs, rot_off=16)
    for _ in range(2):
        src.copy_(torch.as_tensor(g.standard_normal((n, 2, 96)).astype(np.float32)))
        pos.copy_(_t(g.integers(0, 1 << 30, size=n).astype(np.int32)))
        gr.replay()
        torch.cuda.synchronize()
        want = O.rope_rows(_f64(src), np_(pos), freqs.numpy(), 1.0, 16)
        assert (np.abs(_f64(dst) - want) <= _bound(_f64(src), want, 1.0, torch.float32)).all()


def test_rows_past_4_gib():
    hs = lib()
    g = np.random.default_rng(7)
    n = (1 << 32) // 1152 + 100
    cache = torch.zeros((n, 576), dtype=torch.bfloat16, device=DEV)
    src = torch.as_tensor(g.standard_normal((50, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    slots = (n - 1 - g.permutation(90)[:50]).astype(np.int32)
    pos = g.integers(0, 1 << 20, size=50).astype(np.int32)
    freqs, _ = hs.hs_rope_freqs(64)
    hs.hs_rope_rows(src, cache, _t(pos), freqs.to(DEV), rot_off=512, dst_slots=_t(slots))
    x = _f64(src)
    want = O.rope_rows(x[:, None], pos, freqs.numpy(), 1.0, 512)[:, 0]
    assert (np.abs(_f64(cache[_t(slots.astype(np.int64))]) - want) <= _bound(x, want, 1.0, torch.bfloat16)).all()
    assert not cache[:1000].any()


def test_refusals():
    hs = lib()
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    freqs = hs.hs_rope_freqs(64)[0].to(DEV)
    for bad in (lambda: hs.hs_rope_rows(x, x.float(), pos, freqs), lambda: hs.hs_rope_rows(x, x[:, :1], pos, freqs),
                lambda: hs.hs_rope_rows(x, x[:, :, :32], pos, freqs), lambda: hs.hs_rope_rows(x, x, pos[:3], freqs),
                lambda: hs.hs_rope_rows(x, x[:3], pos, freqs), lambda: hs.hs_rope_rows(x, x.cpu(), pos, freqs),
                lambda: hs.hs_rope_rows(x, x, pos, freqs, dst_slots=pos[:2]), lambda: hs.hs_rope_rows(x, x, pos, freqs[None]),
                lambda: hs.hs_rope_rows(x.transpose(1, 2), x, pos, freqs), lambda: hs.hs_rope_rows(x, x, pos.long(), freqs),
                lambda: hs.hs_rope_rows(x.half(), x.half(), pos, freqs), lambda: hs.hs_rope_rows(x, x, pos, freqs.cpu())):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (lambda: hs.hs_rope_rows(x, x, pos, freqs, rot_off=1), lambda: hs.hs_rope_rows(x, x, pos, freqs, layout=2),
                lambda: hs.hs_rope_rows(x, x, pos, freqs, factor=float("inf")),
                lambda: hs.hs_rope_rows(x, x[:1].expand(4, 2, 64), pos, freqs)):
        with pytest.raises(hs.HisparseError):
            bad()
