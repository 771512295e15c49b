"""Sampled verification with noise at the ends of the float range: it counts as
within [2^-126, 2^126]. Every request's decisions are clear of rounding (the
oracle's margins say so), and all are compared."""
import math

import numpy as np
import pytest
import torch

from oracle import hs_oracle as O
from gpu_util import lib, np_
from test_gpu_verify_sample import _case, _check, _run, _t

pytestmark = pytest.mark.gpu
DEV = "cuda"
TINY, HUGE = np.float32(1e-40), np.float32(3e38)


def _all(hs, c):
    want = O.verify_sample(*c)
    assert (want[3] > 2.0 ** -16).all()
    got = _run(hs, *c)
    _check(got, want)
    return got


def _noisy(kind, E, g):
    B, V = E.shape
    if kind == "one tiny":
        E[np.arange(B), g.integers(0, V, B)] = TINY
    elif kind == "many tiny":
        E[g.random(E.shape) < 0.3] = TINY
    elif kind == "all tiny":
        E[:] = TINY
    elif kind == "all huge":
        E[:] = HUGE
    elif kind == "all infinite":
        E[:] = math.inf
    elif kind == "huge beside large":
        E[:] = np.where(g.random(E.shape) < 0.5, HUGE, np.float32(2.0 ** 125))
    elif kind == "huge where it matters":
        E[g.random(E.shape) < 0.7] = HUGE
    elif kind == "ends":
        E[:] = np.where(g.random(E.shape) < 0.5, np.float32(2.0 ** -126), np.float32(2.0 ** 126))
    return E


KINDS = ["one tiny", "many tiny", "all tiny", "all huge", "all infinite", "huge beside large",
         "huge where it matters", "ends"]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("B,d,V", [(4, 2, 96), (3, 2, 1001), (2, 1, 20000)])
@pytest.mark.parametrize("kind", KINDS)
def test_noise_at_the_ends(kind, B, d, V, probs, dtype):
    hs = lib()
    seed = V + 7 * KINDS.index(kind) + 1000 * probs
    for k in range(50):                                    # a seed whose decisions are all clear
        c = _case(seed + 100000 * k, B, d, V, dtype, probs)
        _noisy(kind, c[5], np.random.default_rng(seed + 1))
        if (O.verify_sample(*c)[3] > 2.0 ** -16).all():
            break
    got = _all(hs, c)
    assert (got[1] >= 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_noise_at_the_ends_of_arrays_off_sixteen_bytes(dtype):
    hs = lib()
    B, V = 3, 5000
    for kind in ("many tiny", "all huge", "huge beside large"):
        c = _case(6, B, 0, V, dtype, False)
        _noisy(kind, c[5], np.random.default_rng(2))
        want = O.verify_sample(*c)
        assert (want[3] > 2.0 ** -16).all()
        flat = torch.empty(B * V + 1, device=DEV)
        E = flat[1:].view(B, V)
        E.copy_(_t(c[5]))
        acc = torch.empty(B, dtype=torch.int32, device=DEV)
        nxt, lp = torch.empty_like(acc), torch.empty((B, 1), device=DEV)
        hs.hs_verify_sample(c[0].to(DEV), _t(c[1]), None, None, None, E, acc, nxt, logprob=lp)
        _check((np_(acc), np_(nxt), np_(lp)), want)


def test_tiny_noise_beside_an_infinite_logit():
    """The infinite logit counts as the largest finite one, its noise as it is."""
    hs = lib()
    B, d, V = 4, 0, 300
    for dtype in (torch.float32, torch.bfloat16):
        logits, T, x, _, u, E = _case(9, B, d, V, dtype, False)
        logits[0, 0, 7] = math.inf                         # all the weight is its own
        E[0, 3] = TINY
        logits[1, 0, 7] = logits[1, 0, 200] = math.inf     # two, told apart by their noise
        E[1, 7], E[1, 200] = 1.0, 0.5
        logits[2, 0, 7] = logits[2, 0, 200] = math.inf
        E[2, 7], E[2, 200] = 1.0, TINY
        logits[3, 0, 7] = logits[3, 0, 200] = math.inf
        E[3, 7], E[3, 200] = HUGE, np.float32(2.0 ** 124)
        got = _run(hs, logits, T, x, None, u, E)
        assert got[1].tolist() == [7, 200, 200, 200]
        assert O.verify_sample(logits, T, x, None, u, E)[1].tolist() == [7, 200, 200, 200]


@pytest.mark.parametrize("B,d,V", [(1, 3, 40000), (2, 5, 3000), (60, 3, 20000)])
def test_inputs_overwritten_during_the_call(B, d, V):
    """Temperatures, numbers and drafts change while calls run: which of them a
    call takes is not said, but all warps of a request take the same, so that
    every call ends, with an answer of its range, and later ones are right."""
    hs = lib()
    c = _case(77, B, d, V, torch.bfloat16, True)
    other = _case(78, B, d, V, torch.bfloat16, True)
    logits, (T, x, q, u, E) = c[0].to(DEV), [_t(a) for a in c[1:]]
    nT, nx, nu = _t(other[1]), _t(other[2]), _t(other[4])
    nT[::2] = 0.0
    acc = torch.empty((40, B), dtype=torch.int32, device=DEV)
    nxt = torch.empty_like(acc)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(40):
        hs.hs_verify_sample(logits, T, x, q, u, E, acc[k], nxt[k])
        with torch.cuda.stream(side):
            for a, b in ((T, nT), (x, nx), (u, nu)):
                t = a.clone()
                a.copy_(b)
                b.copy_(t)
    torch.cuda.synchronize()
    assert int(acc.min()) >= 0 and int(acc.max()) <= d and int(nxt.min()) >= 0 and int(nxt.max()) < V
    for a, b in zip((T, x, u), (c[1], c[2], c[4])):
        a.copy_(_t(b))
    got = torch.empty(B, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
    hs.hs_verify_sample(logits, T, x, q, u, E, *got)
    _check((np_(got[0]), np_(got[1]), None), O.verify_sample(*c))
