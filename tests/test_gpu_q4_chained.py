"""The 4-bit cache and the rotary positions behind the calls that write what they
read, with no wait of the host between them; rows and parts of one tile; the first
calls of a process and of a thread."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import hs_oracle as O
from gpu_util import lib
from test_gpu_q4 import _attend, _cache, _check, _f64, _indices, _q, _space, _t

pytestmark = pytest.mark.gpu
DEV = "cuda"
REPEATS = 30


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("H", [128, 20, 16])
def test_every_step_sees_its_own_values(H, split):
    """Indices from hs_resolve_topk (which lets the attention start beside it),
    rows rotated and quantised, q rotated in place right before the attention:
    every call must see its own step's values, in places that held an earlier
    step's."""
    hs = lib()
    g = np.random.default_rng(19 + H)
    B, L, bs, K, steps = 4, 900, 64, 300, 8
    nblk = (L + bs) // bs + 1
    n = B * nblk * bs
    bt = g.permutation(B * nblk).reshape(B, nblk).astype(np.int32)
    clen, req = np.full(B, L, np.int32), np.arange(B, dtype=np.int32)
    d_req, d_clen, d_bt = _t(req), _t(clen), _t(bt)
    freqs, _ = hs.hs_rope_freqs(64)
    d_freqs = freqs.to(DEV)
    rows = [g.standard_normal((n, 576)).astype(np.float32) for _ in range(steps)]
    pos = [g.integers(0, 100000, size=n).astype(np.int32) for _ in range(steps)]
    topks = [np.stack([g.permutation(L)[:K] for _ in range(B)]).astype(np.int32) for _ in range(steps)]
    qs = [_q(g, B, H) for _ in range(steps)]
    d_rows, d_pos, d_topks, d_qs = [_t(r) for r in rows], [_t(p) for p in pos], [_t(t) for t in topks], [q.to(DEV) for q in qs]
    cache = torch.zeros((n, 416), dtype=torch.uint8, device=DEV)
    turned, q = torch.zeros((n, 576), device=DEV), torch.zeros((B, H, 576), dtype=torch.bfloat16, device=DEV)
    q_pos = _t(clen - 1)
    topk = torch.zeros((B, K), dtype=torch.int32, device=DEV)
    idx = torch.zeros_like(topk)
    ws = _space() if split else None
    outs = [torch.empty((B, H, 512), dtype=torch.bfloat16, device=DEV) for _ in range(steps)]
    lses = [torch.empty((B, H), device=DEV) for _ in range(steps)]
    twice, kept_q, kept = [torch.empty_like(o) for o in outs], [], []
    torch.cuda.synchronize()
    for s in range(steps):
        topk.copy_(d_topks[s])
        q.copy_(d_qs[s])
        hs.hs_rope_rows(q, q, q_pos, d_freqs, rot_off=512)
        hs.hs_rope_rows(d_rows[s], turned, d_pos[s], d_freqs, rot_off=512)
        hs.hs_quant_rows_q4(turned, cache)
        hs.hs_resolve_topk(d_req, d_clen, d_bt, topk, bs, bs, idx)
        hs.hs_sparse_attn_decode_q4(q, cache, idx, 1 / 24, outs[s], lse=lses[s], workspace=ws)
        kept_q.append(q.clone())
        kept.append(turned.clone())
        # what the attention reads, written by the kernels right before it
        hs.hs_quant_rows_q4(d_rows[(s + 1) % steps], cache)
        hs.hs_quant_rows_q4(turned, cache)
        q.copy_(d_qs[s])
        hs.hs_rope_rows(q, q, q_pos, d_freqs, rot_off=512)
        hs.hs_sparse_attn_decode_q4(q, cache, idx, 1 / 24, twice[s], workspace=ws)
    torch.cuda.synchronize()
    for s in range(steps):
        e_idx, _, _ = O.resolve_topk(req, clen, bt, topks[s], bs, bs)
        values = O.q4_values(O.q4_quantise(_f64(kept[s])))
        _check(outs[s], lses[s], _f64(kept_q[s]), values, e_idx, 1 / 24)
        assert torch.equal(outs[s], twice[s])
        want = O.rope_rows(_f64(qs[s]), clen - 1, freqs.numpy(), 1.0, 512)
        assert (np.abs(_f64(kept_q[s]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * np.abs(_f64(qs[s])).max()).all()


@pytest.mark.parametrize("kind", ["bf16", "q8", "q4"])
def test_attention_right_behind_the_rotation_of_its_queries(kind):
    """Many times over: queries of another step rotated in place, attended over at
    once."""
    hs = lib()
    g = np.random.default_rng(31)
    R, H, K, n = 96, 128, 64, 2000
    x = torch.as_tensor(g.standard_normal((n, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    if kind == "bf16":
        kv, call = x, hs.hs_sparse_attn_decode
    elif kind == "q8":
        kv, call = torch.zeros((n, 656), dtype=torch.uint8, device=DEV), hs.hs_sparse_attn_decode_q8
        hs.hs_quant_rows(x, kv)
    else:
        kv, call = torch.zeros((n, 416), dtype=torch.uint8, device=DEV), hs.hs_sparse_attn_decode_q4
        hs.hs_quant_rows_q4(x, kv)
    idx = _t(_indices(g, R, K, n, 0.0))
    freqs = hs.hs_rope_freqs(64)[0].to(DEV)
    raw = [_q(g, R, H).to(DEV) for _ in range(4)]
    pos = [_t(g.integers(0, 1 << 20, size=R).astype(np.int32)) for _ in range(4)]
    want = []
    for r, p in zip(raw, pos):
        q = r.clone()
        hs.hs_rope_rows(q, q, p, freqs, rot_off=512)
        torch.cuda.synchronize()
        out = torch.empty((R, H, 512), dtype=torch.bfloat16, device=DEV)
        call(q, kv, idx, 1 / 24, out)
        torch.cuda.synchronize()
        want.append(out)
    q = torch.empty_like(raw[0])
    got = [torch.empty_like(want[0]) for _ in range(40)]
    for k in range(40):
        # (every dim of q comes through the call)
        hs.hs_rope_rows(raw[k % 4], q, pos[k % 4], freqs, rot_off=512)
        call(q, kv, idx, 1 / 24, got[k])
    torch.cuda.synchronize()
    for k in range(40):
        assert torch.equal(got[k], want[k % 4])


@pytest.mark.parametrize("R,H,K", [(1, 128, 1), (2, 17, 32), (5, 128, 31), (90, 128, 32), (200, 130, 20), (400, 64, 7)])
def test_rows_of_one_tile(R, H, K):
    """One CTA of the pair then owns no tile, and takes the other's P over a place
    where its own Q has landed."""
    hs = lib()
    g = np.random.default_rng(R * 1009 + H * 7 + K)
    rows, values = _cache(g, 500)
    idx = _indices(g, R, K, 500, 0.1)
    idx[0, 0] = 3
    q = _q(g, R, H)
    dq, cache, di = q.to(DEV), _t(rows), _t(idx)
    out, lse = _attend(hs, dq, cache, di, 1 / 24)
    _check(out, lse, _f64(q), values, idx, 1 / 24)
    for _ in range(REPEATS):
        again, lse2 = _attend(hs, dq, cache, di, 1 / 24)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("R,H,K", [(1, 128, 672), (1, 17, 670), (2, 128, 653), (1, 256, 1313), (1, 16, 2049), (3, 5, 97)])
def test_a_last_part_of_one_tile(R, H, K):
    """21 tiles in parts of 5, 5, 5, 5 and 1 (42: 5 x 8, 2), with a workspace."""
    hs = lib()
    g = np.random.default_rng(R * 1013 + H * 7 + K)
    rows, values = _cache(g, 900)
    idx = _indices(g, R, K, 900, 0.05)
    q = _q(g, R, H)
    ws, cache, dq, di = _space(), _t(rows), q.to(DEV), _t(idx)
    out, lse = _attend(hs, dq, cache, di, 1 / 24, ws)
    _check(out, lse, _f64(q), values, idx, 1 / 24)
    for _ in range(REPEATS):
        again, lse2 = _attend(hs, dq, cache, di, 1 / 24, ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


SETUP = """
import threading
import torch
import hisparse_top_sparse_gb300 as hs
d = "cuda"
g = torch.Generator(device=d).manual_seed(1)
src = torch.randn((400, 576), device=d, generator=g).bfloat16()
cache = torch.zeros((400, 416), dtype=torch.uint8, device=d)
back = torch.zeros_like(src)
heads = [128, 16, 40, 128, 16, 5]
q = [torch.randn((3, h, 576), device=d, generator=g).bfloat16() for h in heads]
idx = [torch.randint(-1, 400, (3, 600), dtype=torch.int32, device=d, generator=g) for _ in heads]
ws = [torch.empty(hs.ATTN_Q4_WORKSPACE_BYTES, dtype=torch.uint8, device=d) for _ in heads]
pos = torch.arange(400, dtype=torch.int32, device=d)
freqs = hs.hs_rope_freqs(64)[0].to(d)
outs = lambda: [torch.zeros((3, h, 512), dtype=torch.bfloat16, device=d) for h in heads]
turned = [torch.zeros_like(src) for _ in range(3)]
torch.cuda.synchronize()
"""

CAPTURED = SETUP + """
def run(o, t):
    hs.hs_rope_rows(src, t, pos, freqs, rot_off=512)
    hs.hs_quant_rows_q4(t, cache)
    hs.hs_dequant_rows_q4(cache, back)
    for i in range(2):
        hs.hs_sparse_attn_decode_q4(q[i], cache, idx[i], 0.04, o[i], workspace=ws[i])


a, b = outs(), outs()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    run(a, turned[0])
gr.replay()
run(b, turned[1])
torch.cuda.synchronize()
assert torch.equal(turned[0], turned[1]) and back.abs().sum() > 0
for i in range(2):
    assert torch.equal(a[i], b[i]) and a[i].abs().sum() > 0
"""

NEW_THREAD = SETUP + """
hs.hs_quant_rows_q4(src, cache)
CALLS = dict(
    quant=lambda o, t, s: hs.hs_quant_rows_q4(src, cache, stream=s),
    dequant=lambda o, t, s: hs.hs_dequant_rows_q4(cache, back, stream=s),
    many=lambda o, t, s: hs.hs_sparse_attn_decode_q4(q[0], cache, idx[0], 0.04, o[0], workspace=ws[0], stream=s),
    few=lambda o, t, s: hs.hs_sparse_attn_decode_q4(q[1], cache, idx[1], 0.04, o[1], workspace=ws[1], stream=s),
    rope=lambda o, t, s: hs.hs_rope_rows(src, t, pos, freqs, rot_off=512, stream=s))
call = CALLS["{call}"]
here, there = outs(), outs()
side = torch.cuda.Stream().cuda_stream
torch.cuda.synchronize()
call(here, turned[0], side)
torch.cuda.synchronize()
bad = []


def work():
    try:
        call(there, turned[1], side)
    except BaseException as e:
        bad.append(e)


t = threading.Thread(target=work)
t.start()
t.join(120)
assert not bad, bad
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(here, there)) and torch.equal(turned[0], turned[1])
"""

THREADS = SETUP + """
hs.hs_quant_rows_q4(src, cache)
N = len(heads)
streams = [torch.cuda.Stream() for _ in heads]
start = threading.Barrier(N)
a, b = outs(), outs()
t = [torch.zeros_like(src) for _ in heads]
bad = []
torch.cuda.synchronize()


def work(i):
    try:
        start.wait(60)
        for _ in range(20):
            hs.hs_sparse_attn_decode_q4(q[i], cache, idx[i], 0.04, a[i], workspace=ws[i], stream=streams[i])
            hs.hs_rope_rows(src, t[i], pos, freqs, rot_off=512, stream=streams[i])
    except BaseException as e:
        bad.append(e)


threads = [threading.Thread(target=work, args=(i,)) for i in range(N)]
[x.start() for x in threads]
[x.join(120) for x in threads]
torch.cuda.synchronize()
assert not bad, bad
for i in range(N):
    hs.hs_sparse_attn_decode_q4(q[i], cache, idx[i], 0.04, b[i], workspace=ws[i])
    torch.cuda.synchronize()
    assert torch.equal(a[i], b[i]) and a[i].abs().sum() > 0 and torch.equal(t[i], t[0])
"""


@pytest.mark.parametrize("name", ["captured", "threads", "quant", "dequant", "many", "few", "rope"])
def test_first_calls_of_a_process_and_of_a_thread(name):
    lib()
    src = dict(captured=CAPTURED, threads=THREADS).get(name) or NEW_THREAD.replace("{call}", name)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", src], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
