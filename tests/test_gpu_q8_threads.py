"""A process's first attention calls made by several threads at once, each on a
stream and with a workspace of its own: what the library looks up once per
device may be looked up by any of them."""
import os
import subprocess
import sys

import pytest

from gpu_util import lib

pytestmark = pytest.mark.gpu

THREADS = """
import threading
import torch
import hisparse_top_sparse_gb300 as hs
d = "cuda"
hs.lib()
g = torch.Generator(device=d).manual_seed(1)
src = torch.randn((400, 576), device=d, generator=g).bfloat16()
cache = torch.zeros((400, 656), dtype=torch.uint8, device=d)
hs.hs_quant_rows(src, cache)
N = 6
heads = [128, 128, 16, 40, 16, 128]
q = [torch.randn((3, h, 576), device=d, generator=g).bfloat16() for h in heads]
idx = [torch.randint(-1, 400, (3, 600), dtype=torch.int32, device=d, generator=g) for _ in heads]
ws = [torch.empty(hs.ATTN_Q8_WORKSPACE_BYTES, dtype=torch.uint8, device=d) for _ in heads]
outs = [[torch.zeros((3, h, 512), dtype=torch.bfloat16, device=d) for h in heads] for _ in range(3)]
streams = [torch.cuda.Stream() for _ in heads]
start = threading.Barrier(N)
bad = []
torch.cuda.synchronize()


def call(i, out, wide):
    s = streams[i].cuda_stream
    hs.hs_sparse_attn_decode_q8(q[i], cache, idx[i], 0.04, out, workspace=ws[i], stream=s)
    hs.hs_sparse_attn_decode(q[i], src, idx[i], 0.04, wide, stream=s)


def work(i):
    try:
        start.wait(60)
        for _ in range(20):
            call(i, outs[0][i], outs[2][i])
    except BaseException as e:
        bad.append(e)


threads = [threading.Thread(target=work, args=(i,)) for i in range(N)]
[t.start() for t in threads]
[t.join(120) for t in threads]
torch.cuda.synchronize()
assert not bad, bad
for i in range(N):
    wide = torch.zeros_like(outs[2][i])
    call(i, outs[1][i], wide)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][i], outs[1][i]) and torch.equal(outs[2][i], wide) and outs[0][i].abs().sum() > 0
"""


def test_the_first_calls_of_a_process_from_several_threads():
    lib()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", THREADS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
