"""Queries written by the kernel right before an attention call, by whatever kernel,
with no wait of the host between them: every call must see its own step's, in a
place that held an earlier step's."""
import numpy as np
import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = ["bf16", "mixed", "q8", "q4"]
R, K, N = 96, 64, 2000


def _call(hs, kind, g):
    """The attention of a kind over its own cache and indices: a function of (q, out)."""
    x = torch.as_tensor(g.standard_normal((N, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    idx = torch.as_tensor(g.integers(0, N, size=(R, K)).astype(np.int32), device=DEV)
    if kind == "bf16":
        return lambda q, out: hs.hs_sparse_attn_decode(q, x, idx, 1 / 24, out)
    if kind == "mixed":
        req = torch.arange(R, dtype=torch.int32, device=DEV)
        resident = (req % 2).to(torch.int32)
        hot = x.flip(0).contiguous()
        return lambda q, out: hs.hs_sparse_attn_decode_mixed(q, x, hot, req, resident, idx, 1 / 24, out)
    row, quant, attend = ((656, hs.hs_quant_rows, hs.hs_sparse_attn_decode_q8) if kind == "q8" else
                          (416, hs.hs_quant_rows_q4, hs.hs_sparse_attn_decode_q4))
    kv = torch.zeros((N, row), dtype=torch.uint8, device=DEV)
    quant(x, kv)
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    return lambda q, out: attend(q, kv, idx, 1 / 24, out, workspace=ws)


def _queries(g, H):
    return [torch.as_tensor(g.standard_normal((R, H, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV) for _ in range(4)]


def _waited(call, qs):
    """What each of the queries gives on its own, all that it reads long in place."""
    want = []
    for q in qs:
        out = torch.zeros((*q.shape[:2], 512), dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        call(q, out)
        torch.cuda.synchronize()
        want.append(out)
    assert not torch.equal(want[0], want[1])
    return want


def _writers(qs, q):
    """Kernels that write step k's queries into q, as a program would."""
    wide = [x.float() for x in qs]
    rows = torch.cat([x.reshape(R, -1) for x in qs])
    at = [torch.arange(R, device=DEV) + k * R for k in range(4)]
    # (products with a unit matrix: exactly the queries)
    unit = torch.eye(576, dtype=torch.bfloat16, device=DEV)
    flat = q.view(-1, 576)
    return {
        "copy": lambda k: q.copy_(qs[k]),
        "cast": lambda k: q.copy_(wide[k]),
        "gather": lambda k: torch.index_select(rows, 0, at[k], out=q.view(R, -1)),
        "product": lambda k: torch.mm(qs[k].view(-1, 576), unit, out=flat),
    }


@pytest.mark.parametrize("H", [128, 24, 16])
@pytest.mark.parametrize("kind", KINDS)
def test_queries_written_by_ordinary_kernels(kind, H):
    hs = lib()
    g = np.random.default_rng(41 + H)
    call, qs = _call(hs, kind, g), _queries(g, H)
    want = _waited(call, qs)
    q = torch.zeros_like(qs[0])
    for name, write in _writers(qs, q).items():
        got = [torch.zeros_like(want[0]) for _ in range(40)]
        write(0)
        torch.cuda.synchronize()
        for k in range(40):
            write(k % 4)
            call(q, got[k])
        torch.cuda.synchronize()
        for k in range(40):
            assert torch.equal(got[k], want[k % 4]), (name, k)


@pytest.mark.parametrize("kind", KINDS)
def test_queries_written_inside_a_graph(kind):
    hs = lib()
    g = np.random.default_rng(43)
    call, qs = _call(hs, kind, g), _queries(g, 128)
    want = _waited(call, qs)
    q = torch.zeros_like(qs[0])
    write = _writers(qs, q)
    got = [torch.zeros_like(want[0]) for _ in range(12)]
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        for k in range(12):
            write["copy" if k % 2 else "cast"](k % 4)
            call(q, got[k])
    for _ in range(5):
        for out in got:
            out.zero_()
        gr.replay()
        torch.cuda.synchronize()
        for k in range(12):
            assert torch.equal(got[k], want[k % 4]), k


@pytest.mark.parametrize("H", [128, 24, 16])
@pytest.mark.parametrize("kind", KINDS)
def test_queries_written_by_a_kernel_that_lets_the_attention_start_beside_it(kind, H):
    """hs_resolve_topk releases what comes behind it as it begins. Its indices are
    32-bit words of the caller's choosing (one block a request, so that a position is
    its own row): here two bf16 values each, the next step's queries, which eight
    of its blocks take some hundreds of microseconds to write. An attention that reads
    q as it starts would see the step before."""
    hs = lib()
    g = np.random.default_rng(47 + H)
    call, qs = _call(hs, kind, g), _queries(g, H)
    for q in qs:
        q[..., 1::2].abs_()               # the high halves: positions are not negative
    want = _waited(call, qs)
    bs, rows = 1 << 20, 8
    req = torch.zeros(rows, dtype=torch.int32, device=DEV)
    clen = torch.full((rows,), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
    bt = torch.arange(2048, dtype=torch.int32, device=DEV)[None].contiguous()
    words = [q.view(torch.int32).reshape(rows, -1) for q in qs]
    assert all(int(w.min()) >= 0 and int(w.max()) < 2 ** 31 - 1 for w in words)
    q = torch.zeros_like(qs[0])
    to = q.view(torch.int32).reshape(rows, -1)
    got = [torch.zeros_like(want[0]) for _ in range(12)]
    torch.cuda.synchronize()
    for k in range(12):
        hs.hs_resolve_topk(req, clen, bt, words[k % 4], bs, bs, to)
        call(q, got[k])
    torch.cuda.synchronize()
    assert torch.equal(q, qs[11 % 4])
    for k in range(12):
        assert torch.equal(got[k], want[k % 4]), k
