"""GPU parity of the sampled verification (hs_verify_sample and its commit)
against the float64 oracle."""
import math

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


def _case(seed, B, d, V, dtype, probs, masked=0.0, spread=2.5):
    g = np.random.default_rng(seed)
    l = g.standard_normal((B, d + 1, V)) * spread
    if masked:
        cut = g.random(l.shape) < masked
        cut[:, :, V // 2] = False
        l[cut] = -np.inf
    logits = torch.as_tensor(l.astype(np.float32)).to(dtype)
    T = (0.5 + g.random(B)).astype(np.float32)
    draft = l[:, :d] + g.standard_normal((B, d, V)) * 0.6
    z = np.exp(draft / T[:, None, None] - (draft / T[:, None, None]).max(-1, keepdims=True))
    q = (z / z.sum(-1, keepdims=True)).astype(np.float32)
    x = (q / g.exponential(size=q.shape)).argmax(-1) if probs else draft.argmax(-1)
    return (logits, T, x.astype(np.int32), q if probs else None, g.random((B, d)).astype(np.float32),
            np.maximum(g.exponential(size=(B, V)), 1e-30).astype(np.float32))


def _run(hs, logits, T, x, q, u, E, logprob=True, status=None):
    B, d1, _ = logits.shape
    acc = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    nxt = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    lp = torch.full((B, d1), 77.0, device=DEV) if logprob else None
    hs.hs_verify_sample(logits.to(DEV), _t(T), _t(x), None if q is None else _t(q), _t(u), _t(E), acc, nxt,
                        logprob=lp, status=status)
    return np_(acc), np_(nxt), np_(lp) if logprob else None


def _check(got, want):
    """Whole numbers equal wherever no decision compared two numbers within
    2^-16 of each other (f32 sums and exponentials are within 2^-17, see the
    log-probabilities); those: ln p = x - ln S, x rounded twice in f32, S
    a tree of at most V / 4096 + 30 additions (2^-24 each) of terms off by
    2^-22 and by their argument's rounding (30 * 2^-24 at weights that
    matter): 2^-17 in all."""
    acc, nxt, lp = got
    e_acc, e_nxt, e_lp, margin = want
    clear = margin > 2.0 ** -16
    assert clear.mean() >= 0.95 or clear.sum() >= len(clear) - 1
    assert np.array_equal(acc[clear], e_acc[clear])
    assert np.array_equal(nxt[clear], e_nxt[clear])
    if lp is not None:
        a, e = lp[clear].astype(np.float64), e_lp[clear]
        inf = np.isinf(e)
        assert np.array_equal(a[inf], e[inf])
        assert (np.abs(a - e)[~inf] <= 2.0 ** -17 + 2.0 ** -21 * np.abs(e[~inf])).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("B,d,V,masked", [(1, 0, 1, 0.0), (3, 1, 2, 0.0), (2, 3, 1024, 0.0), (5, 4, 1001, 0.5),
                                           (40, 2, 333, 0.95), (1, 7, 50257, 0.0), (3, 15, 9999, 0.2),
                                           (2, 3, 129280, 0.0), (160, 2, 4097, 0.1), (330, 1, 700, 0.0),
                                           (2, 40, 100, 0.0), (1, 255, 64, 0.0), (2000, 1, 40, 0.2),
                                           (1, 3, 40000, 0.0), (9, 3, 32768, 0.0), (70, 5, 20000, 0.9),
                                           (3, 2, 50259, 0.0), (20, 3, 12346, 0.3), (300, 1, 2570, 0.0),
                                           (110, 3, 30004, 0.0), (4, 3, 515, 0.6)])
def test_against_the_oracle(dtype, probs, B, d, V, masked):
    hs = lib()
    c = _case(B * 131 + d * 17 + V, B, d, V, dtype, probs, masked)
    c[1][::3] = 0.0                                        # some greedy requests among them
    got = _run(hs, *c)
    _check(got, O.verify_sample(*c))
    again = _run(hs, *c)
    assert all(np.array_equal(a, b) for a, b in zip(got, again))
    acc, nxt, _ = _run(hs, *c, logprob=False)
    assert np.array_equal(acc, got[0]) and np.array_equal(nxt, got[1])


def test_every_length_is_accepted():
    """Uniforms that accept exactly m drafts of each request, m = 0..d."""
    hs = lib()
    d, V = 6, 5003
    B = d + 1
    logits, T, x, q, u, E = _case(5, B, d, V, torch.bfloat16, True)
    u[:] = 0.0
    q[q == 0] = 1e-9
    for m in range(d):
        u[m, m] = 1.0
        q[m, m, x[m, m]] = 1e6                             # refused whatever p is
    got = _run(hs, logits, T, x, q, u, E)
    want = O.verify_sample(logits, T, x, q, u, E)
    assert np.array_equal(got[0], np.arange(d + 1))
    _check(got, want)


def test_greedy_requests_equal_the_greedy_call():
    hs = lib()
    for V, dtype in [(1000, torch.float32), (129, torch.bfloat16), (4099, torch.float32), (129280, torch.bfloat16)]:
        B, d = 6, 3
        g = np.random.default_rng(V)
        lg = torch.as_tensor(g.integers(-3, 4, size=(B, d + 1, V)).astype(np.float32)).to(dtype)   # many ties
        x = lg.float().numpy()[:, :d].argmax(-1).astype(np.int32)
        x[1, 0] += 1
        x[2, 2] += 1
        acc = torch.empty(B, dtype=torch.int32, device=DEV)
        nxt = torch.empty_like(acc)
        hs.hs_verify_accept_noalloc(lg.to(DEV), _t(x), acc, nxt)
        for T in (0.0, -1.0, float("nan")):
            a, n, _ = _run(hs, lg, np.full(B, T, np.float32), x, None, np.ones((B, d), np.float32),
                           np.ones((B, V), np.float32))
            assert np.array_equal(a, np_(acc)) and np.array_equal(n, np_(nxt))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [7, 1003, 20000])
def test_masked_infinite_and_absent_logits(dtype, V):
    hs = lib()
    B, d = 8, 2
    logits, T, x, q, u, E = _case(V, B, d, V, dtype, True)
    logits[0] = -math.inf                                  # nothing left in the first row
    logits[1, 1] = float("nan")                            # nothing left in the second
    u[1, 0] = 0.0
    logits[2, 0, ::2] = float("nan")
    logits[3, 0, 3] = math.inf
    logits[4, 0, 1::2] = -math.inf
    logits[5] = -math.inf
    T[5] = 0.0                                             # greedy, nothing left
    logits[6, :, 2] = math.inf
    T[6] = 0.0
    logits[7, 0] = 1e38 * torch.sign(logits[7, 0].float()).to(dtype)
    got = _run(hs, logits, T, x, q, u, E)
    _check(got, O.verify_sample(logits, T, x, q, u, E))
    assert got[1][0] == -1 and got[1][5] == -1 and got[1][6] == 2


def test_temperatures_of_every_size():
    hs = lib()
    temps = np.array([1e-42, 1e-30, 1e-6, 1e-3, 0.1, 1.0, 30.0, 1e4, 1e30, np.inf], np.float32)
    B, d, V = len(temps), 2, 801
    logits, _, x, q, u, E = _case(3, B, d, V, torch.float32, True, masked=0.1)
    # the smallest differences, so that tiny temperatures leave one token and huge ones all
    with np.errstate(over="ignore"):
        got = _run(hs, logits, temps, x, q, u, E)
        want = O.verify_sample(logits, temps, x, q, u, E)
    clear = want[3] > 2.0 ** -16
    assert clear.sum() >= B - 1
    assert np.array_equal(got[0][clear], want[0][clear]) and np.array_equal(got[1][clear], want[1][clear])


def test_drafts_outside_the_vocabulary_and_an_empty_residual():
    hs = lib()
    B, d, V = 4, 2, 300
    logits, T, x, q, u, E = _case(11, B, d, V, torch.float32, True)
    u[:] = 0.0
    x[0, 0], x[1, 1], x[2, 0] = V, -1, 2 ** 30
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    for probs in (q, None):
        st.zero_()
        got = _run(hs, logits, T, x, probs, u, E, status=st)
        assert int(st.item()) == hs.HS_STATUS_INDEX
        assert got[0][0] == 0 and got[0][1] <= 1 and got[0][2] == 0
        _check(got, O.verify_sample(logits, T, x, probs, u, E))
    # draft "probabilities" above the target's everywhere: the target's own are drawn from
    x[:] = 5
    u[:] = 1.0
    got = _run(hs, logits, T, x, np.full_like(q, 2.0), u, E)
    assert not got[0].any()
    _check(got, O.verify_sample(logits, T, x, np.full_like(q, 2.0), u, E))


def test_unaligned_rows_and_a_captured_replay():
    hs = lib()
    B, d, V = 3, 3, 2047
    logits, T, x, q, u, E = _case(21, B, d, V, torch.bfloat16, True)
    flat = torch.empty(logits.numel() + 3, dtype=torch.bfloat16, device=DEV)
    off = flat[3:].view(B, d + 1, V)                       # six bytes off
    off.copy_(logits)
    dev = [_t(a) for a in (T, x, q, u, E)]
    acc = torch.empty(B, dtype=torch.int32, device=DEV)
    nxt, lp = torch.empty_like(acc), torch.empty((B, d + 1), device=DEV)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        hs.hs_verify_sample(off, *dev, acc, nxt, logprob=lp)
    for seed in (21, 22, 23):
        c = _case(seed, B, d, V, torch.bfloat16, True)
        off.copy_(c[0])
        for t, a in zip(dev, c[1:]):
            t.copy_(_t(a))
        gr.replay()
        torch.cuda.synchronize()
        _check((np_(acc), np_(nxt), np_(lp)), O.verify_sample(*c))


def test_two_streams_at_once():
    hs = lib()
    cases = [_case(31 + i, 5, 3, 30011, torch.bfloat16, True) for i in range(2)]
    dev = [[c[0].to(DEV)] + [_t(a) for a in c[1:]] for c in cases]
    outs = [(torch.empty(5, dtype=torch.int32, device=DEV), torch.empty(5, dtype=torch.int32, device=DEV)) for _ in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for args, o, s in zip(dev, outs, streams):
            hs.hs_verify_sample(*args, *o, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        _check((np_(o[0]), np_(o[1]), None), O.verify_sample(*c))


def _buffer(hs, B, S, n_step, max_ctx, bs, extra=0):
    pool = torch.zeros(((B + extra) * max_ctx, 576), dtype=torch.bfloat16).pin_memory()
    hot = torch.zeros(((B + extra) * (S + n_step), 576), dtype=torch.bfloat16, device=DEV)
    n = (B + extra) * (max_ctx // bs)
    hbt = np.random.default_rng(0).permutation(n).astype(np.int32).reshape(B + extra, -1)
    buf = hs.HsBuffer(B + extra, S, n_step, max_ctx, bs, hot, pool, _t(hbt))
    return buf, O.HotBuffer(B + extra, S, n_step, max_ctx, bs, hbt, pool.clone()), hot, pool


@pytest.mark.parametrize("seed", range(3))
def test_finalize_commits_the_accepted_prefix(seed):
    """Several steps on scattered request ids, one request at its context's
    end: results, maps, hot rows, host rows and status against the oracle."""
    hs = lib()
    g = np.random.default_rng(50 + seed)
    B, d, V, S, bs, max_ctx = 4, 3, 500, 9, 4, 48
    buf, ref, hot, pool = _buffer(hs, B, S, d + 1, max_ctx, bs, extra=3)
    L = g.integers(0, 20, size=B + 3).astype(np.int32)
    kv_len = _t(L.copy())
    for step in range(4):
        ids = g.permutation(B + 3)[:B].astype(np.int32)
        if step == 3:
            L[ids[0]] = max_ctx                              # no room left: refused, reported
            kv_len.copy_(_t(L))
        c = _case(seed * 10 + step, B, d, V, torch.float32, seed % 2 == 0)
        c[4][0] = 0.0
        skv = W.bf16_normal((B, d + 1, 576), 1.0, seed * 10 + step, "skv")
        acc = torch.empty(B, dtype=torch.int32, device=DEV)
        nxt, lp = torch.empty_like(acc), torch.empty((B, d + 1), device=DEV)
        q = None if c[3] is None else _t(c[3])
        hs.hs_verify_sample_finalize(buf, c[0].to(DEV), _t(c[1]), _t(c[2]), q, _t(c[4]), _t(c[5]), skv.to(DEV),
                                     kv_len, acc, nxt, logprob=lp, req_ids=_t(ids))
        e = O.verify_sample(*c)
        assert (e[3] > 2.0 ** -16).all()
        _check((np_(acc), np_(nxt), np_(lp)), e)
        ref.now += 1
        bits = skv.view(torch.int16).numpy().view(np.uint16)
        st = 0
        for k, b in enumerate(ids):
            if ref.commit(int(b), int(L[b]), bits[k, :e[0][k] + 1], ref.now):
                L[b] += e[0][k] + 1
            else:
                st |= O.STATUS_CAPACITY
        assert np.array_equal(np_(kv_len), L) and hs.hs_get_status(buf) == st
        assert (step == 3) == (st != 0)
        ts, stok, sts = buf.dump()
        for b in range(B + 3):
            assert np.array_equal(ts[b].numpy(), ref.token_slot_array(b))
        assert np.array_equal(hot.view(torch.int16).cpu().numpy().view(np.uint16), ref.hot)
        assert np.array_equal(pool.view(torch.int16).numpy().view(np.uint16), ref.host_pool)
    buf.close()


def test_finalize_refusals():
    hs = lib()
    B, d, V = 2, 1, 64
    buf, _, _, _ = _buffer(hs, B, 4, d + 1, 16, 4)
    logits, T, x, q, u, E = _case(1, B, d, V, torch.float32, True)
    dev = [logits.to(DEV)] + [_t(a) for a in (T, x, q, u, E)]
    skv = torch.zeros((B, d + 1, 576), dtype=torch.bfloat16, device=DEV)
    kv_len = torch.zeros(B, dtype=torch.int32, device=DEV)
    acc = torch.empty(B, dtype=torch.int32, device=DEV)
    nxt = torch.empty_like(acc)
    with pytest.raises(ValueError):
        hs.hs_verify_sample_finalize(buf, *dev, skv[:, :1].contiguous(), kv_len, acc, nxt)
    with pytest.raises(ValueError):
        hs.hs_verify_sample_finalize(buf, *dev, skv, kv_len[:1], acc, nxt)
    with pytest.raises(TypeError):
        hs.hs_verify_sample_finalize(buf, dev[0], dev[1].double(), *dev[2:], skv, kv_len, acc, nxt)
    clock = buf.clock
    three = [_t(a) for a in _case(1, 3, d, V, torch.float32, True)[1:]]
    with pytest.raises(hs.HisparseError):                   # more requests than the buffer serves
        hs.hs_verify_sample_finalize(buf, torch.zeros((3, d + 1, V), device=DEV), *three,
                                     torch.zeros((3, d + 1, 576), dtype=torch.bfloat16, device=DEV), kv_len,
                                     torch.empty(3, dtype=torch.int32, device=DEV),
                                     torch.empty(3, dtype=torch.int32, device=DEV))
    assert buf.clock == clock
    # a repeated request commits once
    ids = torch.zeros(B, dtype=torch.int32, device=DEV)
    hs.hs_verify_sample_finalize(buf, *dev, skv, kv_len, acc, nxt, req_ids=ids)
    assert hs.hs_get_status(buf) == hs.HS_STATUS_INDEX
    assert int(kv_len[0]) in ((np_(acc) + 1).tolist()) and int(kv_len[1]) == 0
    # a captured commit is refused, on the capturing stream, with nothing enqueued
    s = torch.cuda.Stream()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        with pytest.raises(hs.HisparseError) as err:
            hs.hs_verify_sample_finalize(buf, *dev, skv, kv_len, acc, nxt)
        acc.add_(0)
    assert err.value.code == hs.HS_ERR_UNSUPPORTED
    buf.close()


@pytest.mark.parametrize("shift", ["logits", "probs", "noise"])
def test_one_array_off_its_sixteen_bytes(shift):
    """A vocabulary of whole 16-byte vectors whose arrays do not all start on
    one: the same answers as aligned ones."""
    hs = lib()
    B, d, V = 4, 2, 4096
    logits, T, x, q, u, E = _case(41, B, d, V, torch.bfloat16, True)
    dev = {"logits": logits.to(DEV), "probs": _t(q), "noise": _t(E)}
    flat = torch.empty(dev[shift].numel() + 1, dtype=dev[shift].dtype, device=DEV)
    off = flat[1:].view(dev[shift].shape)
    off.copy_(dev[shift])
    dev[shift] = off
    acc = torch.empty(B, dtype=torch.int32, device=DEV)
    nxt, lp = torch.empty_like(acc), torch.empty((B, d + 1), device=DEV)
    hs.hs_verify_sample(dev["logits"], _t(T), _t(x), dev["probs"], _t(u), dev["noise"], acc, nxt, logprob=lp)
    _check((np_(acc), np_(nxt), np_(lp)), O.verify_sample(logits, T, x, q, u, E))


def test_equal_ratios_go_to_the_lowest_index():
    """Uniform logits and noise: every token is drawn alike."""
    hs = lib()
    for V in (5, 1000, 4096, 131072):
        for dtype in (torch.float32, torch.bfloat16):
            B, d = 3, 1
            logits = torch.zeros((B, d + 1, V), dtype=dtype)
            u = np.array([[0.0], [1.0], [1.0]], np.float32)
            x = np.array([[V - 1], [0], [V // 2]], np.int32)
            got = _run(hs, logits, np.ones(B, np.float32), x, None, u, np.ones((B, V), np.float32))
            # accepted: the lowest of all; refused: the lowest but the draft's own
            assert got[0].tolist() == [1, 0, 0] and got[1].tolist() == [0, 1, 0]


def test_refusals_of_the_binding():
    hs = lib()
    B, d, V = 2, 1, 64
    logits, T, x, q, u, E = _case(1, B, d, V, torch.float32, True)
    good = dict(logits=logits.to(DEV), temperature=_t(T), draft_tokens=_t(x), draft_probs=_t(q), uniforms=_t(u),
                noise=_t(E), accept_len=torch.empty(B, dtype=torch.int32, device=DEV),
                next_token=torch.empty(B, dtype=torch.int32, device=DEV))
    hs.hs_verify_sample(**good)
    for k, v in (("logits", good["logits"].half()), ("temperature", good["temperature"].double()),
                 ("draft_tokens", good["draft_tokens"].long()), ("noise", good["noise"].bfloat16())):
        with pytest.raises(TypeError):
            hs.hs_verify_sample(**dict(good, **{k: v}))
    for k, v in (("temperature", good["temperature"][:1]), ("draft_probs", good["draft_probs"][:, :, :32]),
                 ("uniforms", good["uniforms"].cpu()), ("noise", good["noise"].t().contiguous().t()),
                 ("uniforms", None), ("noise", None), ("logits", good["logits"].transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            hs.hs_verify_sample(**dict(good, **{k: v}))
    with pytest.raises(hs.HisparseError):
        hs.hs_verify_sample(**{k: (v[:0] if v is not None else None) for k, v in good.items()})
