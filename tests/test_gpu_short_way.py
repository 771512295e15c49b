"""The binding's two ways to a call: one native function that checks and calls,
and, where anything is not plainly what it takes, the checks argument by argument.
Both give the same results and the same refusals."""
import numpy as np
import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _calls(hs, g):
    """(name, function of the arguments that replace its own, those of its outputs)."""
    n = 40
    x = torch.as_tensor(g.standard_normal((n, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    wide = torch.as_tensor(g.standard_normal((n, 640)).astype(np.float32)).to(DEV)[:, 64:]
    slots = torch.as_tensor(g.permutation(60)[:n].astype(np.int32), device=DEV)
    q = torch.as_tensor(g.standard_normal((3, 20, 576)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    idx = torch.as_tensor(g.integers(-1, n, size=(3, 700)).astype(np.int32), device=DEV)
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    freqs = hs.hs_rope_freqs(64)[0].to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = {}
    for fmt, rb in (("", 656), ("_q4", 416)):
        cache = torch.zeros((60, rb), dtype=torch.uint8, device=DEV)
        filled = torch.zeros((n, rb), dtype=torch.uint8, device=DEV)
        getattr(hs, "hs_quant_rows" + fmt)(x, filled)
        back = torch.zeros((n, 576), device=DEV)
        out["quant" + fmt] = (getattr(hs, "hs_quant_rows" + fmt),
                              dict(src=wide, cache=cache, src_slots=None, dst_slots=slots, status=st), cache)
        out["dequant" + fmt] = (getattr(hs, "hs_dequant_rows" + fmt),
                                dict(cache=filled, dst=back, src_slots=pos, dst_slots=None, status=None), back)
        o = torch.zeros((3, 20, 512), dtype=torch.bfloat16, device=DEV)
        out["attend" + fmt] = (getattr(hs, "hs_sparse_attn_decode" + (fmt or "_q8")),
                               dict(q=q, kv=filled, idx=idx, scale=0.05, out=o, lse=torch.zeros((3, 20), device=DEV),
                                    workspace=ws, status=st), o)
    to = torch.zeros((60, 576), dtype=torch.bfloat16, device=DEV)
    out["rope"] = (hs.hs_rope_rows, dict(src=x, dst=to, positions=pos, freqs=freqs, factor=1.5, rot_off=512,
                                         layout=hs.HS_ROPE_HALF, inverse=True, src_slots=None, dst_slots=slots, status=st), to)
    return out


NAMES = ["quant", "dequant", "attend", "quant_q4", "dequant_q4", "attend_q4", "rope"]


@pytest.mark.parametrize("name", NAMES)
def test_both_ways_give_the_same(name, monkeypatch):
    hs = lib()
    assert hs._native is not None, "the binding's native module is not built"
    f, kw, out = _calls(hs, np.random.default_rng(1))[name]
    seen = []
    for native in (hs._native, None):
        monkeypatch.setattr(hs, "_native", native)
        for more in (dict(), dict(stream=torch.cuda.current_stream()), dict(stream=torch.cuda.current_stream().cuda_stream)):
            out.zero_()
            f(**kw, **more)
            seen.append(out.clone())
    torch.cuda.synchronize()
    assert seen[0].float().abs().sum() > 0
    assert all(torch.equal(s, seen[0]) for s in seen)


def _spoilt(kw):
    """The arguments with one of them wrong, in every way that fits its kind."""
    for k, v in kw.items():
        if isinstance(v, torch.Tensor):
            yield k, v.cpu()
            yield k, v.to(torch.float16) if v.is_floating_point() else v.to(torch.int16)
            yield k, v[None]
            yield k, torch.cat([v, v])[::2] if v.dim() == 1 else torch.stack([v, v], -1)[..., 0]
            yield k, "text"
            if k in ("src", "cache", "kv", "q", "idx", "out", "lse", "dst", "positions", "freqs") and v.dim() > 1:
                yield k, v[..., :-1]
            if k in ("positions", "src_slots", "dst_slots", "idx", "out", "lse"):
                yield k, v[:-1]
        elif k in ("scale", "factor"):
            yield k, "text"
            yield k, float("nan")
        elif k == "layout":
            yield k, 7
        elif k == "rot_off":
            yield k, 513
            yield k, 1 << 40


@pytest.mark.parametrize("name", NAMES)
def test_both_ways_refuse_the_same(name, monkeypatch):
    hs = lib()
    f, kw, out = _calls(hs, np.random.default_rng(2))[name]
    native = hs._native
    refused = 0
    for k, v in _spoilt(kw):
        ends = []
        for way in (native, None):
            monkeypatch.setattr(hs, "_native", way)
            out.zero_()
            try:
                f(**dict(kw, **{k: v}))
                ends.append(out.clone())
            except Exception as e:                  # which one is compared
                ends.append((type(e), str(e)))
        if isinstance(ends[0], tuple) or isinstance(ends[1], tuple):
            assert ends[0] == ends[1], (k, ends)
            refused += 1
        else:
            assert torch.equal(ends[0], ends[1]), k
    torch.cuda.synchronize()
    assert refused >= 5
