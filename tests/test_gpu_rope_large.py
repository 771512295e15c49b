"""Rotations as large as those that give a thread eight rows, or more heads of a row
than it has in flight: every element against the oracle, within the bound of the
smaller ones."""
import numpy as np
import pytest
import torch

from oracle import hs_oracle as O
from gpu_util import lib
from test_gpu_rope import _bound, _f64, _freqs, _t

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rotate(hs, src, dst, pos, freqs, factor, off, half, **kw):
    hs.hs_rope_rows(src, dst, _t(pos), freqs.to(DEV), factor=factor, rot_off=off,
                    layout=hs.HS_ROPE_HALF if half else hs.HS_ROPE_INTERLEAVED, **kw)


def _values(g, shape, dtype):
    return torch.as_tensor(g.standard_normal(shape, dtype=np.float32)).to(dtype).to(DEV)


def _oracle(x, pos, freqs, factor, off, half):
    """O.rope_rows of the rotated dims, the others as they are."""
    rot = 2 * len(freqs)
    want = x.copy()
    want[:, :, off:off + rot] = O.rope_rows(x[:, :, off:off + rot], pos, freqs.numpy(), factor, 0, half)
    return want


# rows (none a multiple of eight), heads, dims, offset, rotated, wider source, wider
# destination; the last column: 16-byte accesses, which rotated or wider dims of other
# sizes rule out
FEW_HEADS = [(12345, 1, 576, 512, 64, 0, 0, True), (12345, 1, 576, 512, 64, 0, 1, False), (12346, 2, 192, 128, 64, 64, 64, True),
             (9999, 2, 63, 3, 60, 1, 0, False), (12347, 3, 96, 0, 64, 0, 32, True), (4099, 3, 101, 5, 94, 0, 3, False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,H,dim,off,rot,more_src,more_dst,vector", FEW_HEADS)
def test_eight_rows_a_thread(n, H, dim, off, rot, more_src, more_dst, vector, half, dtype):
    hs = lib()
    g = np.random.default_rng(n * 31 + dim + half)
    src = _values(g, (n, H, dim + more_src), dtype)[:, :, more_src:]
    rows = n + 77
    wide = torch.full((rows, H, dim + more_dst), 7.0, dtype=dtype, device=DEV)
    dst = wide[:, :, more_dst:]
    pos = g.integers(-1000, 1 << 20, size=n).astype(np.int32)
    freqs, factor = _freqs(hs, rot, True)
    # units of 16 bytes or one element (pairs), the rule by which a thread takes eight rows
    per = 16 // src.element_size() if vector else 1
    units = (dim - rot) // per + (rot // per if vector and not half else rot // 2 // per)
    assert n * H * units >= torch.cuda.get_device_properties(0).multi_processor_count * 512 and n % 8
    s = g.integers(0, n, size=n).astype(np.int32)
    d = g.permutation(rows)[:n].astype(np.int32)
    s[::11], d[5::13] = -1, -1                 # no entry
    s[3::101], d[7::97] = n, rows + 3          # past the rows: left out, and told
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    _rotate(hs, src, dst, pos, freqs, factor, off, half, src_slots=_t(s), dst_slots=_t(d), status=st)
    assert int(st.item()) == hs.HS_STATUS_INDEX
    ok = (s >= 0) & (d >= 0) & (s < n) & (d < rows)
    x = _f64(src)
    y = _oracle(x[s[ok]], pos[ok], freqs, factor, off, half)
    got = _f64(wide)
    written = np.zeros(rows, bool)
    written[d[ok]] = True
    assert (got[~written] == 7).all() and (got[:, :, :more_dst] == 7).all()
    z = got[d[ok]][:, :, more_dst:]
    assert (np.abs(z - y) <= _bound(x[s[ok]], y, factor, dtype)).all()
    beside = np.ones(dim, bool)
    beside[off:off + rot] = False
    assert np.array_equal(z[:, :, beside], x[s[ok]][:, :, beside])
    # without lists, and in place: the same bits
    st.zero_()
    plain = torch.full((n, H, dim + more_dst), 7.0, dtype=dtype, device=DEV)
    _rotate(hs, src, plain[:, :, more_dst:], pos, freqs, factor, off, half, status=st)
    y = _oracle(x, pos, freqs, factor, off, half)
    assert (np.abs(_f64(plain[:, :, more_dst:]) - y) <= _bound(x, y, factor, dtype)).all()
    assert (plain[:, :, :more_dst] == 7).all()
    _rotate(hs, src, src, pos, freqs, factor, off, half, status=st)
    assert torch.equal(src, plain[:, :, more_dst:]) and int(st.item()) == 0


# a thread's heads: h, h + step, ... of the row, more than the four in flight (the last
# turn not whole)
MANY_HEADS = [(1501, 65, 64, 0, 64, 0, 0, True), (1200, 128, 80, 8, 64, 16, 0, True), (1503, 61, 66, 1, 64, 0, 1, False),
              (411, 301, 64, 0, 32, 0, 64, True)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,H,dim,off,rot,more_src,more_dst,vector", MANY_HEADS)
def test_more_heads_a_thread_than_it_has_in_flight(n, H, dim, off, rot, more_src, more_dst, vector, half, dtype):
    hs = lib()
    g = np.random.default_rng(n * 37 + dim + half)
    src = _values(g, (n, H, dim + more_src), dtype)[:, :, more_src:]
    wide = torch.full((n + 1, H, dim + more_dst), 7.0, dtype=dtype, device=DEV)
    dst = wide[:n, :, more_dst:]
    pos = g.integers(0, 1 << 20, size=n).astype(np.int32)
    freqs, factor = _freqs(hs, rot, True)
    per = 16 // src.element_size() if vector else 1
    units = (dim - rot) // per + (rot // per if vector and not half else rot // 2 // per)
    each = n * H * units // (torch.cuda.get_device_properties(0).multi_processor_count * 512)
    assert each > 4
    _rotate(hs, src, dst, pos, freqs, factor, off, half)
    x = _f64(src)
    y = _oracle(x, pos, freqs, factor, off, half)
    assert (np.abs(_f64(dst) - y) <= _bound(x, y, factor, dtype)).all()
    assert (wide[n] == 7).all() and (wide[:, :, :more_dst] == 7).all()
    # in place, whole: the same bits (then units are the rotated ones alone)
    _rotate(hs, src, src, pos, freqs, factor, off, half)
    assert torch.equal(src, dst)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,H", [(20000, 1), (2000, 64), (3, 2), (40, 128)])
def test_bits_do_not_depend_on_where_a_row_lies(n, H, half, dtype):
    """Aligned, one element further on, and as rows of a larger call."""
    hs = lib()
    g = np.random.default_rng(n + half)
    x = _values(g, (n, H, 64), dtype)
    pos = g.integers(0, 1 << 20, size=n).astype(np.int32)
    freqs, factor = _freqs(hs, 64, True)
    out = torch.zeros_like(x)
    _rotate(hs, x, out, pos, freqs, factor, 0, half)
    odd = torch.zeros((n, H, 65), dtype=dtype, device=DEV)[:, :, 1:]
    _rotate(hs, x, odd, pos, freqs, factor, 0, half)
    assert torch.equal(out, odd)
    odd.copy_(x)
    _rotate(hs, odd, odd, pos, freqs, factor, 0, half)
    assert torch.equal(out, odd)
    some = torch.zeros((3, H, 64), dtype=dtype, device=DEV)
    _rotate(hs, x[-3:], some, pos[-3:], freqs, factor, 0, half)
    assert torch.equal(out[-3:], some)


def test_a_large_step_of_rows_and_queries_from_prompt_to_cache():
    """Latent rows and queries of one prompt as a program moves them, one call each,
    with the rows' own positions: rotated rows into the slots of a bf16 cache, then a
    second time from the same source, for what a call before it may have left."""
    hs = lib()
    g = np.random.default_rng(8)
    n, rows = 20011, 30000
    freqs, factor = _freqs(hs, 64, True)
    cache = torch.zeros((rows, 576), dtype=torch.bfloat16, device=DEV)
    for turn in range(2):
        src = _values(g, (n, 576), torch.bfloat16)
        slots = g.permutation(rows)[:n].astype(np.int32)
        pos = g.integers(0, 1 << 17, size=n).astype(np.int32)
        before = _f64(cache)
        _rotate(hs, src, cache, pos, freqs, factor, 512, True, dst_slots=_t(slots))
        x = _f64(src)[:, None]
        y = _oracle(x, pos, freqs, factor, 512, True)
        got = _f64(cache)
        assert (np.abs(got[slots][:, None] - y) <= _bound(x, y, factor, torch.bfloat16)).all()
        rest = np.ones(rows, bool)
        rest[slots] = False
        assert np.array_equal(got[rest], before[rest])
