"""Operators of a decode step over a quantised latent cache and of its sampled verification, as measured cases.

Three families, told apart by ``case["op"]``:

* ``write`` / ``read``: latent rows quantised into a cache's slots as they are written, and rows of such a cache read
  back. A row of 576 dims is held in 656 bytes: 512 e4m3 codes, 64 bf16 rope dims, 16 exponents (biased by 127), one
  power of two for each 32 dims.
* ``attn``: attention of decode rows over their selected rows of such a cache (values: the first 512 dims).
* ``verify``: drafted tokens accepted or refused against the target's probabilities with given random numbers.
"""

import math

import torch

own = False

D, DV, ROPE, GROUP, ROW = 576, 512, 64, 32, 656
NG = DV // GROUP
E_MIN, E_MAX = -112, 120
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one request's anchor and three drafts, written each step: the smallest call, where latency counts
        {"name": "write 4 step rows", "op": "write", "n": 4, "cache": 4099, "type": "bf16", "out": "bf16", "width": 576, "skip": 0},
        # a prompt chunk as a projection leaves it (a slice of wider rows), its padding tokens without a slot
        {"name": "write a prompt chunk", "op": "write", "n": 8191, "cache": 65536, "type": "bf16", "out": "bf16", "width": 640, "skip": 37},
        # a resident cache of 32 requests x 8192 positions converted row by row
        {"name": "write a resident cache", "op": "write", "n": 262144, "cache": 264192, "type": "bf16", "out": "bf16", "width": 576, "skip": 0},
        # the selected rows of 64 requests read back for a caller that wants them in bf16
        {"name": "read selected rows", "op": "read", "n": 131072, "cache": 262144, "out": "bf16", "skip": 0},
        # two requests, four rows each, few heads and few keys
        {"name": "attn 8 rows 64 keys", "op": "attn", "R": 8, "H": 16, "K": 64, "cache": 1024, "pad": 0.1, "empty": 0},
        # one request's verify rows: few rows, the whole key list
        {"name": "attn 4 rows", "op": "attn", "R": 4, "H": 128, "K": 2048, "cache": 32768, "pad": 0.0, "empty": 0},
        # a ragged batch: odd sizes, padded lists, a row without keys
        {"name": "attn 43 ragged rows", "op": "attn", "R": 43, "H": 80, "K": 1001, "cache": 50021, "pad": 0.3, "empty": 1},
        # 32 requests, anchor and three drafts each
        {"name": "attn 128 rows", "op": "attn", "R": 128, "H": 128, "K": 2048, "cache": 262144, "pad": 0.0, "empty": 0},
        # 128 requests, anchor and three drafts each: the largest step
        {"name": "attn 512 rows", "op": "attn", "R": 512, "H": 128, "K": 2048, "cache": 524800, "pad": 0.0, "empty": 0},
        # two requests over a small vocabulary, f32 logits
        {"name": "verify 2 x 3 drafts", "op": "verify", "B": 2, "d": 3, "V": 1024, "type": "f32", "probs": True, "masked": 0.0, "greedy": 0},
        # drafts without probabilities (taken greedily by the drafter), some requests greedy themselves, an odd vocabulary
        {"name": "verify 33 x 5 sure drafts", "op": "verify", "B": 33, "d": 5, "V": 50257, "type": "bf16", "probs": False, "masked": 0.2, "greedy": 4},
        # 256 requests, three drafts each, the whole vocabulary
        {"name": "verify 256 x 3 drafts", "op": "verify", "B": 256, "d": 3, "V": 129280, "type": "bf16", "probs": True, "masked": 0.0, "greedy": 16},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "verify", "verify"])
    if op in ("write", "read"):
        n = _spread(rng, 1, 150000)
        cache = n + _spread(rng, 1, 60000)
        case = {"op": op, "n": n, "cache": cache, "out": rng.choice(["bf16", "f32"]), "skip": rng.choice([0, 0, 1, 5]) if n > 8 else 0}
        if op == "write":
            case.update(type=rng.choice(["bf16", "f32"]), width=rng.choice([576, 584, 640, 1152]))
        return case
    if op == "attn":
        H = rng.choice([1, 8, 16, 40, 64, 80, 128, 128, 136])
        K = _spread(rng, 1, 8192)
        R = _spread(rng, 1, max(1, min(512, 512 * 2048 * 128 // (K * max(H, 128)))))
        return {"op": op, "R": R, "H": H, "K": K, "cache": max(K, _spread(rng, 64, 300000)), "pad": rng.choice([0.0, 0.05, 0.5]),
                "empty": rng.choice([0, 0, 1]) if R > 1 else 0}
    V = _spread(rng, 100, 150000)
    d = rng.choice([0, 1, 2, 3, 3, 5, 7])
    B = _spread(rng, 1, max(1, min(256, 256 * 4 * 129280 // ((d + 1) * V))))
    return {"op": op, "B": B, "d": d, "V": V, "type": rng.choice(["bf16", "bf16", "f32"]), "probs": rng.random() < 0.6,
            "masked": rng.choice([0.0, 0.0, 0.3, 0.95]), "greedy": rng.choice([0, 0, B // 4])}


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _latent(n, g, dtype, width=D):
    """Latent rows: dims of unlike sizes, a few of them large, as a compressing projection leaves them."""
    x = torch.randn((n, width), generator=g, device="cuda", dtype=torch.bfloat16 if n * width > (1 << 24) else torch.float32)
    dim = torch.exp(torch.randn((width,), generator=g, device="cuda") * 0.5)
    return x.mul_(dim.to(x.dtype)).to(dtype)


def _distinct(n, rows, g):
    return torch.randperm(rows, generator=g, device="cuda")[:n].to(torch.int32)


def _cache(rows, g):
    """A cache in use: codes of all kinds (none of them NaN), rope dims, exponents near those of latent rows."""
    c = torch.empty((rows, ROW), dtype=torch.uint8, device="cuda")
    c[:, :DV] = (torch.randn((rows, DV), generator=g, device="cuda", dtype=torch.bfloat16) * 96).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    c[:, DV:DV + 2 * ROPE] = torch.randn((rows, ROPE), generator=g, device="cuda", dtype=torch.bfloat16).view(torch.uint8)
    c[:, DV + 2 * ROPE:] = torch.randint(119, 122, (rows, NG), generator=g, device="cuda", dtype=torch.uint8)
    return c


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "write":
        n = case["n"]
        wide = _latent(n, g, DTYPES[case["type"]], case["width"])
        s["src"] = wide[:, case["width"] - D:]  # the latent dims are the last ones of each row
        s["cache"] = torch.zeros((case["cache"], ROW), dtype=torch.uint8, device="cuda")
        s["slots"] = _distinct(n, case["cache"], g)
        if case["skip"]:
            s["slots"][n - case["skip"]:] = -1
        s["out"] = torch.zeros((n, D), dtype=DTYPES[case["out"]], device="cuda")
    elif case["op"] == "read":
        s["cache"] = _cache(case["cache"], g)
        s["slots"] = torch.randint(0, case["cache"], (case["n"],), generator=g, device="cuda", dtype=torch.int32)
        if case["skip"]:
            s["slots"][case["n"] - case["skip"]:] = -1
        s["out"] = torch.zeros((case["n"], D), dtype=DTYPES[case["out"]], device="cuda")
    elif case["op"] == "attn":
        R, H, K = case["R"], case["H"], case["K"]
        s["q"] = torch.randn((R, H, D), generator=g, device="cuda").to(torch.bfloat16)
        s["cache"] = _cache(case["cache"], g)
        idx = torch.randint(0, case["cache"], (R, K), generator=g, device="cuda", dtype=torch.int32)
        if case["pad"]:
            idx[torch.rand((R, K), generator=g, device="cuda") < case["pad"]] = -1
        for r in range(case["empty"]):
            idx[(r * 7 + 1) % R] = -1
        s["idx"] = idx
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.empty((R, H, DV), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((R, H), dtype=torch.float32, device="cuda")
        s["workspace"] = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")  # enough for every size of call
    else:
        B, d, V = case["B"], case["d"], case["V"]
        t = torch.rand((B,), generator=g, device="cuda") * 0.8 + 0.5
        logits = torch.randn((B, d + 1, V), generator=g, device="cuda").mul_(2.5)
        if case["masked"]:  # a caller's own cut of unlikely tokens
            cut = torch.rand((B, d + 1, V), generator=g, device="cuda") < case["masked"]
            cut[:, :, V // 2] = False  # one token is always left
            logits.masked_fill_(cut, -math.inf)
        s["logits"] = logits.to(DTYPES[case["type"]])
        drafter = torch.randn((B, d, V), generator=g, device="cuda").mul_(0.6).add_(logits[:, :d]).div_(t[:, None, None])
        probs = torch.softmax(drafter, dim=-1) if case["probs"] else None
        race = torch.empty((B, d, V), device="cuda").exponential_(generator=g).clamp_(min=1e-30)
        s["drafts"] = ((probs / race) if case["probs"] else drafter).argmax(-1).to(torch.int32)
        s["probs"] = probs
        t[:case["greedy"]] = 0.0
        s["temperature"] = t
        s["uniforms"] = torch.rand((B, d), generator=g, device="cuda")
        s["noise"] = torch.empty((B, V), device="cuda").exponential_(generator=g).clamp_(min=1e-30)
        s["accept"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        s["next"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        s["logprob"] = torch.empty((B, d + 1), dtype=torch.float32, device="cuda")
    return s


# --------------------------------------------------------------- one pass --

def _exp2i(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantised(x):
    """f32 rows [n][576] -> cache rows [n][656]."""
    v = x[:, :DV].reshape(-1, NG, GROUP)
    mant, ex = torch.frexp(v.abs().amax(-1))
    e = torch.where(mant == 0, E_MIN, ex - 9 + (mant > 0.875).to(ex.dtype)).clamp(E_MIN, E_MAX)
    codes = (v * _exp2i(-e)[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return torch.cat([codes.reshape(-1, DV).view(torch.uint8), x[:, DV:].to(torch.bfloat16).view(torch.uint8),
                      (e + 127).to(torch.uint8)], dim=1)


def _values(rows):
    """Cache rows [n][656] -> f32 rows [n][576]."""
    codes = rows[:, :DV].contiguous().view(torch.float8_e4m3fn).float().reshape(-1, NG, GROUP)
    scale = _exp2i(rows[:, DV + 2 * ROPE:].to(torch.int32) - 127)
    rope = rows[:, DV:DV + 2 * ROPE].contiguous().view(torch.bfloat16).float()
    return torch.cat([(codes * scale[:, :, None]).reshape(-1, DV), rope], dim=1)


def _read_back(cache, slots, dtype):
    keep = slots >= 0
    rows = _values(cache[slots.clamp(min=0).long()])
    return torch.where(keep[:, None], rows, 0.0).to(dtype)


def _plain_attn(s):
    idx, scale = s["idx"], s["scale"]
    R, K = idx.shape
    ok = (idx >= 0) & (idx < s["cache"].shape[0])
    kv = _values(s["cache"][idx.clamp(min=0).long().reshape(-1)]).reshape(R, K, D)
    x = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * scale
    x = torch.where(ok[:, None, :], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, kv[:, :, :DV]) / torch.where(total == 0, 1.0, total)
    return out.to(torch.bfloat16), (top + torch.log(total))[..., 0]


def _plain_verify(s):
    # in 64 bits: acceptance and the race compare values that may lie next to each other
    t, drafts, probs = s["temperature"].double(), s["drafts"].long(), s["probs"]
    B, d1, V = s["logits"].shape
    d = d1 - 1
    greedy = t == 0
    x = s["logits"].double() / torch.where(greedy, 1.0, t)[:, None, None]
    top = x.amax(-1, keepdim=True)
    logp = x - (top + torch.log(torch.exp(x - top).sum(-1, keepdim=True)))
    best = s["logits"].argmax(-1)
    px = torch.exp(logp[:, :d]).gather(2, drafts[:, :, None])[:, :, 0]
    qx = probs.gather(2, drafts[:, :, None])[:, :, 0].double() if probs is not None else torch.ones_like(px)
    agree = torch.where(greedy[:, None], drafts == best[:, :d], s["uniforms"].double() * qx < px)
    accept = agree.long().cumprod(1).sum(1)
    rows = torch.arange(B, device=t.device)
    p = torch.exp(logp[rows, accept])
    refused = accept < d
    at = accept.clamp(max=max(d - 1, 0))
    if d == 0:
        rest = p
    elif probs is not None:
        rest = torch.where(refused[:, None], (p - probs[rows, at].double()).clamp(min=0), p)
    else:
        rest = p.clone()
        rest[rows, drafts[rows, at]] = torch.where(refused, 0.0, p[rows, drafts[rows, at]])
    rest = torch.where((rest > 0).any(1, keepdim=True), rest, p)
    token = torch.where(greedy, best[rows, accept], (rest / s["noise"].double()).argmax(1))
    given = torch.cat([drafts, token[:, None]], dim=1)
    where = torch.arange(d1, device=t.device)[None, :]
    given = torch.where(where == accept[:, None], token[:, None], given)
    logprob = torch.where(where <= accept[:, None], logp.gather(2, given[:, :, None])[:, :, 0], 0.0)
    return accept.to(torch.int32), token.to(torch.int32), logprob.float()


def run(s):
    op = s["case"]["op"]
    if own:
        import hisparse_top_sparse_gb300 as hs
        if op == "write":
            hs.hs_quant_rows(s["src"], s["cache"], dst_slots=s["slots"])
            hs.hs_dequant_rows(s["cache"], s["out"], src_slots=s["slots"])
            return s["out"]
        if op == "read":
            hs.hs_dequant_rows(s["cache"], s["out"], src_slots=s["slots"])
            return s["out"]
        if op == "attn":
            hs.hs_sparse_attn_decode_q8(s["q"], s["cache"], s["idx"], s["scale"], s["out"], lse=s["lse"], workspace=s["workspace"])
            return s["out"], s["lse"]
        hs.hs_verify_sample(s["logits"], s["temperature"], s["drafts"], s["probs"], s["uniforms"], s["noise"], s["accept"], s["next"],
                            logprob=s["logprob"])
        return s["accept"], s["next"], s["logprob"]
    if op == "write":
        keep = s["slots"] >= 0
        s["cache"][s["slots"][keep].long()] = _quantised(s["src"].float())[keep]
        return _read_back(s["cache"], s["slots"], s["out"].dtype)
    if op == "read":
        return _read_back(s["cache"], s["slots"], s["out"].dtype)
    if op == "attn":
        return _plain_attn(s)
    return _plain_verify(s)


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "write":  # source rows read, cache rows written, values written
        n = case["n"]
        return {"bytes": n * (D * size[case["type"]] + ROW + D * size[case["out"]] + 4), "flops": 2 * n * D}
    if case["op"] == "read":
        n = case["n"]
        return {"bytes": n * (ROW + D * size[case["out"]] + 4), "flops": n * D}
    if case["op"] == "attn":
        R, H, K = case["R"], case["H"], case["K"]
        keys = K * (1 - case["pad"]) * (R - case["empty"])
        # a cached row read by several rows is read once
        rows = min(keys, case["cache"] * (1 - math.exp(-keys / case["cache"])))
        return {"bytes": rows * ROW + R * (4 * K + H * (2 * D + 2 * DV + 4)), "flops": 2 * keys * H * (D + DV)}
    # the logits up to the first refusal (about two drafts in three pass), one row of draft probabilities and of noise
    B, d, V = case["B"], case["d"], case["V"]
    rows = sum((2 / 3) ** i for i in range(d + 1))
    per = rows * V * size[case["type"]] + 4 * V + (4 * V * (1 - (2 / 3) ** d) if case["probs"] else 0)
    return {"bytes": B * per, "flops": 4 * B * V * (rows + 1)}


# ------------------------------------------------------------ in 64 bits --

def _e4m3(y):
    """The nearest e4m3 value of each y (ties to even), |y| <= 448, in 64 bits."""
    low = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    low = torch.where(torch.exp2(low) > y.abs(), low - 1, low).clamp(min=-6)
    step = torch.exp2(low - 3)
    return torch.round(y / step) * step


def _exact_rows(cache, slots):
    """Values of cache rows from the layout's definition: sign, exponent and fraction of each code taken apart."""
    b = cache[slots].to(torch.int64)
    c = b[:, :DV]
    frac, ex = c & 7, (c >> 3) & 15
    mag = torch.where(ex == 0, frac.double() * 2.0 ** -9, (8 + frac).double() * torch.exp2(ex.double() - 10))
    v = torch.where(c >= 128, -mag, mag) * torch.exp2(b[:, DV + 2 * ROPE:].double() - 127).repeat_interleave(GROUP, 1)
    r = b[:, DV:DV + 2 * ROPE]
    bits = (r[:, 0::2] | (r[:, 1::2] << 8)) << 16
    bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
    return torch.cat([v, bits.view(torch.float32).double()], 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        x, parts = s["src"], []
        for a in range(0, case["n"], 1 << 15):
            y = x[a:a + (1 << 15)].double()
            v = y[:, :DV].reshape(-1, NG, GROUP)
            most = v.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(torch.where(most == 0, 2.0 ** -150, most) / 448))
            e = torch.where(448 * torch.exp2(e - 1) >= most, e - 1, e)
            e = torch.where(448 * torch.exp2(e) < most, e + 1, e).clamp(E_MIN, E_MAX)
            v = (_e4m3(v * torch.exp2(-e)) * torch.exp2(e)).reshape(-1, DV)
            y = torch.cat([v, x[a:a + (1 << 15), DV:].to(torch.bfloat16).double()], 1)
            parts.append(torch.where(s["slots"][a:a + (1 << 15), None] >= 0, y, 0.0))
        return torch.cat(parts)
    if case["op"] == "read":
        parts = []
        for at in s["slots"].long().split(1 << 15):
            parts.append(_exact_rows(s["cache"], at.clamp(min=0)) * (at >= 0)[:, None])
        return torch.cat(parts)
    if case["op"] == "attn":
        outs, lses = [], []
        for r in range(case["R"]):
            at = s["idx"][r]
            at = at[at >= 0].long()
            if at.numel() == 0:
                outs.append(torch.zeros((case["H"], DV), dtype=torch.float64, device="cuda"))
                lses.append(torch.full((case["H"],), -math.inf, dtype=torch.float64, device="cuda"))
                continue
            kv = _exact_rows(s["cache"], at)
            x = (s["q"][r].double() @ kv.T) * s["scale"]
            lses.append(torch.logsumexp(x, 1))
            outs.append(torch.softmax(x, 1) @ kv[:, :DV])
        return torch.stack(outs), torch.stack(lses)
    accept, token, logprob = [], [], []
    for b in range(case["B"]):
        t = float(s["temperature"][b])
        logp = torch.log_softmax(s["logits"][b].double() / (t if t > 0 else 1.0), -1)
        m, d = 0, case["d"]
        while m < d:
            x = int(s["drafts"][b, m])
            if t > 0:
                q = float(s["probs"][b, m, x]) if case["probs"] else 1.0
                if not float(s["uniforms"][b, m]) * q < math.exp(float(logp[m, x])):
                    break
            elif x != int(s["logits"][b, m].argmax()):
                break
            m += 1
        w = torch.exp(logp[m])
        if t == 0:
            x = int(s["logits"][b, m].argmax())
        else:
            if m < d:
                rest = w - s["probs"][b, m].double() if case["probs"] else w.clone()
                if not case["probs"]:
                    rest[int(s["drafts"][b, m])] = 0.0
                w = rest.clamp(min=0) if bool((rest > 0).any()) else w
            x = int((w / s["noise"][b].double()).argmax())
        given = [int(v) for v in s["drafts"][b, :m]] + [x]
        lp = torch.zeros(d + 1, dtype=torch.float64)
        for i, v in enumerate(given):
            lp[i] = float(logp[i, v])
        accept.append(m)
        token.append(x)
        logprob.append(lp)
    return torch.tensor(accept, dtype=torch.int32), torch.tensor(token, dtype=torch.int32), torch.stack(logprob)
