"""Calls of a thread that has made no CUDA call before, in a process whose
other threads have."""
import os
import subprocess
import sys

import pytest

from gpu_util import lib

pytestmark = pytest.mark.gpu

NEW_THREAD = """
import threading
import torch
import hisparse_top_sparse_gb300 as hs
d = "cuda"
g = torch.Generator(device=d).manual_seed(1)
src = torch.randn((400, 576), device=d, generator=g).bfloat16()
cache = torch.zeros((400, 656), dtype=torch.uint8, device=d)
q = torch.randn((3, {H}, 576), device=d, generator=g).bfloat16()
idx = torch.randint(-1, 400, (3, 600), dtype=torch.int32, device=d, generator=g)
ws = torch.empty(hs.ATTN_Q8_WORKSPACE_BYTES, dtype=torch.uint8, device=d)
v = (torch.randn((2, 3, 1000), device=d), torch.ones(2, device=d), torch.zeros((2, 2), dtype=torch.int32, device=d),
     None, torch.zeros((2, 2), device=d), torch.rand((2, 1000), device=d) + 0.1)
back = torch.zeros_like(src)
buf = hs.HsBuffer(2, 4, 3, 32, 4, torch.zeros((14, 576), dtype=torch.bfloat16, device=d),
                  torch.zeros((64, 576), dtype=torch.bfloat16).pin_memory(),
                  torch.arange(16, dtype=torch.int32, device=d).view(2, 8))
step_kv, kv_len = torch.zeros((2, 3, 576), dtype=torch.bfloat16, device=d), torch.zeros(2, dtype=torch.int32, device=d)
CALLS = dict(
    quant=lambda o, t, s: hs.hs_quant_rows(src, cache, stream=s),
    dequant=lambda o, t, s: hs.hs_dequant_rows(cache, back, stream=s),
    q8=lambda o, t, s: hs.hs_sparse_attn_decode_q8(q, cache, idx, 0.04, o, workspace=ws, stream=s),
    bf16=lambda o, t, s: hs.hs_sparse_attn_decode(q, src, idx, 0.04, o, stream=s),
    verify=lambda o, t, s: hs.hs_verify_sample(*v, t[0], t[1], stream=s),
    finalize=lambda o, t, s: hs.hs_verify_sample_finalize(buf, *v, step_kv, kv_len, t[0], t[1], stream=s))
call = CALLS["{call}"]
hs.hs_quant_rows(src, cache)
mk = lambda: (torch.zeros((3, {H}, 512), dtype=torch.bfloat16, device=d), torch.full((2, 2), -7, dtype=torch.int32, device=d))
here, there = mk(), mk()
side = torch.cuda.Stream().cuda_stream
call(*here, side)
torch.cuda.synchronize()
bad = []


def work():
    try:
        call(*there, side)
    except BaseException as e:
        bad.append(e)


t = threading.Thread(target=work)
t.start()
t.join(120)
assert not bad, bad
torch.cuda.synchronize()
assert torch.equal(here[0], there[0]) and torch.equal(here[1], there[1])
"""


@pytest.mark.parametrize("call,H", [("quant", 1), ("dequant", 1), ("q8", 128), ("q8", 16), ("bf16", 128), ("verify", 1),
                                    ("finalize", 1)])
def test_the_first_call_of_a_new_thread(call, H):
    lib()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = NEW_THREAD.replace("{H}", str(H)).replace("{call}", call)
    r = subprocess.run([sys.executable, "-c", src], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
