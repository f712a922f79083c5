"""The paged-cache operators as measured work: appending, decoding one token, attending with many new tokens.

``run`` has two forms of each: the framework's calls, and a plain form in elementary torch
operations in 32 bits.  ``exact`` is the definition in 64 bits, sequence by sequence.
A case is one call; its lengths follow from the case alone, its values from the seed.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BASE = 10000.0


def _case(name, op, B, H, Hkv, d, dtype, page, lo, hi, new_lo=1, new_hi=1, cache="16", rot=0,
          interleaved=False, window=0):
    c = {"op": op, "B": B, "H": H, "Hkv": Hkv, "d": d, "dtype": dtype, "page": page, "lo": lo,
         "hi": hi, "new_lo": new_lo, "new_hi": new_hi, "cache": cache, "rot": rot,
         "interleaved": interleaved, "window": window}
    if name:
        c["name"] = name
    return c


def listed():
    """lo..hi: keys of a sequence after the call; new_lo..new_hi: its new tokens among them."""
    return [
        # the append of one generated token of one user: pure latency
        _case("append step b1 bf16", "append", 1, 32, 8, 128, "bf16", 64, 1000, 1000, rot=128),
        # a decoding step of a full batch into E4M3 pages
        _case("append step b64 e4m3", "append", 64, 32, 8, 128, "bf16", 64, 100, 4000, rot=128,
              cache="e4m3"),
        # prompts of odd lengths of a small model, half the columns rotated, pairs interleaved
        _case("append prompts d64 fp16", "append", 8, 16, 16, 64, "fp16", 16, 200, 1500, 100, 1024,
              rot=32, interleaved=True),
        # a large prefill step: 16 prompts of about a thousand tokens
        _case("append prompts d128 bf16", "append", 16, 32, 8, 128, "bf16", 64, 1100, 3000, 600,
              1100, rot=128),
        # one user's token of a small model on a short context: pure latency
        _case("decode b1 n777 d64 fp16", "decode", 1, 16, 16, 64, "fp16", 16, 777, 777),
        # the framework's own decoding benchmark, its caches in pages
        _case("decode b16 kv32k bf16", "decode", 16, 32, 8, 128, "bf16", 64, 16384, 32768),
        # the same from E4M3 pages
        _case("decode b16 kv32k e4m3", "decode", 16, 32, 8, 128, "bf16", 64, 16384, 32768,
              cache="e4m3"),
        # one user far into a long document: few rows, the length has to be split
        _case("decode b1 kv130k bf16", "decode", 1, 32, 8, 128, "bf16", 128, 130049, 130049),
        # a busy server: many ragged sequences, groups of three heads, sliding window, odd pages
        _case("decode b128 ragged window", "decode", 128, 12, 4, 128, "bf16", 20, 1, 4000,
              window=1024),
        # five drafted tokens of four users checked against their contexts
        _case("fwd b4 draft5 bf16", "fwd", 4, 32, 8, 128, "bf16", 64, 1500, 2500, 5, 5),
        # chunks of two long prompts on what is cached of them
        _case("fwd b2 chunk2k kv8k bf16", "fwd", 2, 32, 8, 128, "bf16", 64, 8000, 8192, 2048, 2048),
        # ragged prompts of a small model with a sliding window on small pages
        _case("fwd b8 ragged d64 window", "fwd", 8, 16, 16, 64, "fp16", 16, 300, 3000, 40, 1000,
              window=512),
    ]


HEADS = [(32, 8), (16, 16), (32, 32), (12, 4), (8, 1), (12, 2), (16, 4), (64, 8)]
PAGES = [16, 16, 32, 64, 64, 128, 256, 8, 20, 40]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "decode", "fwd"])
        H, Hkv = rng.choice(HEADS)
        d = rng.choice([32, 64, 128, 128])
        dtype, page = rng.choice(["bf16", "fp16"]), rng.choice(PAGES)
        window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        cache = "e4m3" if d == 128 and op != "fwd" and rng.random() < 0.4 else "16"
        if op == "append":
            step = rng.random() < 0.5
            B = _log(rng, 1, 256 if step else 32)
            new_hi = 1 if step else _log(rng, 2, 4096)
            new_lo = 1 if step else rng.randint(1, new_hi)
            hi = new_hi + _log(rng, 1, 4000)
            lo = rng.randint(new_hi, hi)
            c = _case("", op, B, H, Hkv, d, dtype, page, lo, hi, new_lo, new_hi, cache,
                      rng.choice([0, 32, d, d]), rng.random() < 0.4)
            if sum(_plan(c)[1]) <= 16384 and B * hi <= 1 << 18:
                return c
        elif op == "decode":
            B = _log(rng, 1, 256)
            hi = _log(rng, 1, 131072)
            lo = rng.randint(1, hi)
            c = _case("", op, B, H, Hkv, d, dtype, page, lo, hi, cache=cache, window=window)
            if B * hi * Hkv * d * (1 if cache == "e4m3" else 2) <= 16 * 32768 * 8 * 128 * 2:
                return c
        else:
            B = _log(rng, 1, 16)
            new_hi = _log(rng, 1, 2048)
            new_lo = rng.randint(1, new_hi)
            hi = new_hi + _log(rng, 1, 8192)
            lo = rng.randint(new_hi, hi)
            c = _case("", op, B, H, Hkv, d, dtype, page, lo, hi, new_lo, new_hi, window=window)
            if B * new_hi * hi * H * d <= 2 * 2048 * 8192 * 32 * 128:
                return c


def _plan(case):
    """Lengths of the B sequences and their numbers of new tokens: spread over their ranges by
    the golden ratio's multiples, so neighbours differ."""
    def spread(lo, hi, k):
        return [lo + int((hi - lo) * ((i * 0.6180339887498949 + k) % 1.0) + 0.5)
                for i in range(case["B"])]
    lens = spread(case["lo"], case["hi"], 0.37)
    new = [min(a, n) for a, n in zip(spread(case["new_lo"], case["new_hi"], 0.71), lens)]
    return lens, new


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B, H, Hkv, d, page = (case[k] for k in ("B", "H", "Hkv", "d", "page"))
    t = TYPES[case["dtype"]]
    lens, new = _plan(case)
    T = sum(new)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(t)

    # a pool of pages somewhat larger than what is in use, handed out in random order;
    # the table holds -1 where a sequence has no page yet
    used = [-(-n // page) for n in lens]
    P, width = sum(used) + 3, max(used) + 1
    ids = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    held = torch.tensor(used, device="cuda")
    at = torch.cumsum(held, 0) - held
    slot = torch.arange(width, device="cuda")
    table = torch.where(slot < held[:, None], ids[(at[:, None] + slot).clamp(max=P - 1)],
                        torch.full((), -1, device="cuda", dtype=torch.int32))
    s = {"case": case, "table": table, "scale": 1.0 / math.sqrt(d), "window": case["window"],
         "lens": torch.tensor(lens, device="cuda", dtype=torch.int32), "max_new": max(new),
         "cu": torch.tensor([sum(new[:i]) for i in range(B + 1)], device="cuda",
                            dtype=torch.int32)}
    # 8-bit caches: N(0, 1) values stay below 6, which the scale puts near the largest code
    s["k_scale"], s["v_scale"] = 6.0 / 448.0, 5.5 / 448.0
    for name in ("kc", "vc"):
        x = normal(P, Hkv, page, d)
        if case["cache"] == "e4m3":
            x = (x.float() / s[name[0] + "_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s[name] = x
    if case["op"] == "append":
        # keys and values as one projection gives them: a row of all their heads a token
        kv = normal(T, 2 * Hkv, d)
        s["q"], s["k"], s["v"] = normal(T, H, d), kv[:, :Hkv], kv[:, Hkv:]
        s["q_out"] = torch.empty((T, H, d), device="cuda", dtype=t)
        if case["rot"]:
            r = case["rot"]
            w = BASE ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
            a = torch.arange(max(lens), device="cuda", dtype=torch.float64)[:, None] * w
            s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        else:
            s["cos_sin"] = None
    else:
        s["q"] = normal(B if case["op"] == "decode" else T, H, d)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, H) if case["op"] == "decode" else (H, T), device="cuda",
                               dtype=torch.float32)
    return s


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import exact_io_aware_22_gb300 as fa
    c = s["case"]
    if c["op"] == "append":
        cu = None if c["new_hi"] == 1 else s["cu"]
        if c["cache"] == "e4m3":
            fa.append_paged_fp8(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"],
                                s["k_scale"], s["v_scale"], cu_seqlens=cu, cos_sin=s["cos_sin"],
                                interleaved=c["interleaved"], q=s["q"], q_out=s["q_out"])
        else:
            fa.append_paged(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"],
                            cu_seqlens=cu, cos_sin=s["cos_sin"], interleaved=c["interleaved"],
                            q=s["q"], q_out=s["q_out"])
        return s["q_out"], s["kc"], s["vc"]
    if c["op"] == "decode":
        if c["cache"] == "e4m3":
            return fa.decode_paged_fp8(s["q"], s["kc"], s["vc"], s["table"], s["lens"],
                                       s["k_scale"], s["v_scale"], scale=s["scale"],
                                       window=s["window"], out=s["out"], lse=s["lse"])
        return fa.decode_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"], scale=s["scale"],
                               window=s["window"], out=s["out"], lse=s["lse"])
    return fa.fwd_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["cu"], s["max_new"],
                        scale=s["scale"], window=s["window"], out=s["out"], lse=s["lse"])


# ------------------------------------------------------------------ the plain forms
def _tokens(s):
    """Sequence, index among its new tokens and key position of every new token."""
    cu = s["cu"].long()
    tok = torch.arange(s["q"].shape[0], device="cuda")
    b = (tok[:, None] >= cu[None, 1:]).sum(1)
    return b, tok - cu[b], s["lens"].long()[b] - (cu[b + 1] - tok)


def _turn(x, s, pos):
    c, x = s["case"], x.float()
    r = c["rot"]
    if not r:
        return x
    cs = s["cos_sin"][pos][:, None]
    cos, sin = cs[..., : r // 2], cs[..., r // 2:]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_append(s):
    c = s["case"]
    b, _, pos = _tokens(s)
    at = s["table"].long()[b, pos // c["page"]]
    row = pos % c["page"]
    k, v = _turn(s["k"], s, pos), s["v"].float()
    if c["cache"] == "e4m3":
        k = (k * (1.0 / s["k_scale"])).clamp(-448, 448)
        v = (v * (1.0 / s["v_scale"])).clamp(-448, 448)
    for cache, x in ((s["kc"], k), (s["vc"], v)):
        x = x.to(cache.dtype)
        if c["cache"] == "e4m3":
            cache, x = cache.view(torch.uint8), x.view(torch.uint8)
        cache[at, :, row] = x
    s["q_out"].copy_(_turn(s["q"], s, pos))
    return s["q_out"], s["kc"], s["vc"]


def _cached(s, name):
    """(B, Hkv, width * page, d) of one cache in 32 bits, through the page table."""
    c, x = s["case"], s[name]
    at = s["table"].clamp(min=0).long()
    x = x.view(torch.uint8)[at].view(x.dtype) if c["cache"] == "e4m3" else x[at]
    x = x.transpose(1, 2).flatten(2, 3).float()
    return x * s[name[0] + "_scale"] if c["cache"] == "e4m3" else x


def _softmax_v(score, allowed, v):
    """Output and log-sum-exp of rows of scores over the allowed keys."""
    score = torch.where(allowed, score, torch.full((), -math.inf, device="cuda"))
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - m)
    l = p.sum(-1, keepdim=True)
    return (p @ v) / l, (m + torch.log(l))[..., 0]


def _plain_decode(s):
    c = s["case"]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    k, v = _cached(s, "kc"), _cached(s, "vc")
    score = (s["q"].float().view(B, Hkv, H // Hkv, d) @ k.transpose(2, 3)) * s["scale"]
    j = torch.arange(k.shape[2], device="cuda")
    n = s["lens"][:, None]
    allowed = (j < n) & (j >= (n - s["window"] if s["window"] else 0))
    o, lse = _softmax_v(score, allowed[:, None, None], v)
    return o.reshape(B, H, d).to(s["q"].dtype), lse.reshape(B, H)


def _plain_fwd(s):
    c = s["case"]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    b, i, pos = _tokens(s)
    k, v = _cached(s, "kc"), _cached(s, "vc")
    q = torch.zeros((B, s["max_new"], H, d), device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, -1, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4)
    score = (q @ k.transpose(2, 3)[:, :, None]) * s["scale"]
    at = torch.zeros((B, s["max_new"]), device="cuda", dtype=torch.int64)
    at[b, i] = pos
    j = torch.arange(k.shape[2], device="cuda")
    allowed = j <= at[..., None]
    if s["window"]:
        allowed = allowed & (j > at[..., None] - s["window"])
    o, lse = _softmax_v(score, allowed[:, None, None], v[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(B, -1, H, d)[b, i]
    return o.to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(B, -1, H)[b, i].t().contiguous()


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "decode": _plain_decode, "fwd": _plain_fwd}[
        state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    H, Hkv, d, rot = case["H"], case["Hkv"], case["d"], case["rot"]
    lens, new = _plan(case)
    T, elem = sum(new), 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        # q, k and v read, q and both caches' new rows written, a row of angles for each token
        return {"bytes": T * d * (4 * H + 2 * Hkv * (2 + elem)) + T * rot * 4, "flops": 0}
    w = case["window"]
    if case["op"] == "decode":
        keys = sum(min(n, w) if w else n for n in lens)
        return {"bytes": keys * Hkv * d * 2 * elem + case["B"] * H * (4 * d + 4),
                "flops": 4 * keys * H * d}
    keys = pairs = 0
    for n, m in zip(lens, new):
        keys += min(n, m - 1 + w) if w else n
        full = max(0, n - max(n - m, w)) if w else 0   # queries that see a whole window
        a = m - full                                   # the others, at positions n - m ...
        pairs += full * w + a * (n - m + 1) + a * (a - 1) // 2
    return {"bytes": keys * Hkv * d * 2 * elem + T * H * (4 * d + 4), "flops": 4 * pairs * H * d}


# ------------------------------------------------------------------ the definition, 64 bits
def _exact_turn(x, s, pos):
    r = s["case"]["rot"]
    y = x.double().clone()
    if r:
        cs = s["cos_sin"].double()[pos]
        for i in range(r // 2):
            a, b = (2 * i, 2 * i + 1) if s["case"]["interleaved"] else (i, i + r // 2)
            cos, sin = cs[:, i, None], cs[:, r // 2 + i, None]
            y[..., a] = x[..., a].double() * cos - x[..., b].double() * sin
            y[..., b] = x[..., b].double() * cos + x[..., a].double() * sin
    return y


def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _plan(case)
    page, H, Hkv, d = case["page"], case["H"], case["Hkv"], case["d"]
    eight = case["cache"] == "e4m3"
    if case["op"] == "append":
        kc, vc = s["kc"].double(), s["vc"].double()
        q = torch.empty(s["q"].shape, device="cuda", dtype=torch.float64)
        t0 = 0
        for b, (n, m) in enumerate(zip(lens, new)):
            pos = torch.arange(n - m, n, device="cuda")
            at, row, tok = s["table"][b].long()[pos // page], pos % page, slice(t0, t0 + m)
            kc[at, :, row] = _exact_turn(s["k"][tok], s, pos) / (s["k_scale"] if eight else 1.0)
            vc[at, :, row] = s["v"][tok].double() / (s["v_scale"] if eight else 1.0)
            q[tok] = _exact_turn(s["q"][tok], s, pos)
            t0 += m
        return q, kc, vc
    decode = case["op"] == "decode"
    o = torch.empty(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.empty(s["lse"].shape, device="cuda", dtype=torch.float64)
    t0 = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        at = s["table"][b, : -(-n // page)].long()
        tok = slice(t0, t0 + m)
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        hidden = (j > pos) | ((j <= pos - s["window"]) if s["window"] else False)
        for h in range(Hkv):
            k, v = (s[x][:, h].double()[at].reshape(-1, d)[:n] if not eight else
                    s[x][:, h].view(torch.uint8)[at].view(s[x].dtype).reshape(-1, d)[:n].double()
                    * s[x[0] + "_scale"] for x in ("kc", "vc"))
            for g in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                x = (s["q"][tok, g].double() @ k.t()) * s["scale"]
                x = x.masked_fill(hidden, -math.inf)
                top = x.max(1, keepdim=True).values
                e = (x - top).exp()
                z = e.sum(1, keepdim=True)
                o[tok, g] = (e / z) @ v
                if decode:
                    lse[tok, g] = (top + z.log())[:, 0]
                else:
                    lse[g, tok] = (top + z.log())[:, 0]
        t0 += m
    return o, lse
