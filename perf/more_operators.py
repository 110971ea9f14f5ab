"""The operators of the attention half of a rebuilt layer: sizes to measure them
at, their plain forms, and their definitions in 64 bits.

  rotary   rotation of pairs of a head's values by position, in the interleaved
           or the half layout, over the whole head or its first part, with
           frequencies scaled for long contexts; and its gradient.
  pages    block tables, slot maps and positions of a batch's new tokens, from
           the requests' lengths and a stack of free pages, on the GPU.
  append   queries and keys rotated, keys and values written to their pages, in
           bf16 or in e4m3 with a power of two per row.
  attend   attention of each request's new tokens over its pages: single
           tokens, chunks, whole prompts, mixed; several query heads to a head
           of keys.

Sizes: the OLMoE stack's attention (q, k, v, o of 2048 x 2048; 16 heads of 128),
and generic ones around it: grouped heads, heads of 64, 80 and 96, pages of 16 to
256 tokens and of odd sizes.
"""
import math

import torch

own = False

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
BIAS = 127                    # of the exponents of e4m3 rows
LOWEST, HIGHEST = -100, 119   # of those exponents


# ---------------------------------------------------------------- the cases

def listed():
    whole = {"head_dim": 128, "part": 128, "interleaved": False, "factor": 1.0}
    stack = {"q_heads": 16, "kv_heads": 16, "head_dim": 128}
    return [
        # one token of a serving step, queries and keys side by side: latency
        {"name": "rotary, 1 token", "op": "rotary", "tokens": 1, "heads": 32, **whole},
        # a training batch of 8 sequences of 2048
        {"name": "rotary, 16384 tokens", "op": "rotary", "tokens": 16384, "heads": 32, **whole},
        # the gradient of a ragged batch: pairs side by side, half of each head, a long context
        {"name": "rotary gradient, 10007 tokens", "op": "rotary gradient", "tokens": 10007,
         "heads": 20, "head_dim": 96, "part": 48, "interleaved": True, "factor": 8.0},
        # a step of a small serving batch: one new token each
        {"name": "pages, 8 requests", "op": "pages", "requests": 8, "new": 1, "cached": 4000,
         "page": 16, "short": False},
        # prompts and chunks arriving for a large batch
        {"name": "pages, 200 requests", "op": "pages", "requests": 200, "new": 80,
         "cached": 4000, "page": 32, "short": False},
        # a step of a serving batch
        {"name": "append, 24 tokens", "op": "append", "tokens": 24, "page": 64, "e4m3": False,
         "by_head": True, "part": 128, "interleaved": False, **stack},
        # a prompt's chunk into 8-bit pages, grouped heads
        {"name": "append 8-bit, 8192 tokens", "op": "append", "tokens": 8192, "page": 32,
         "e4m3": True, "by_head": False, "part": 64, "interleaved": False, "q_heads": 32,
         "kv_heads": 8, "head_dim": 128},
        # one token of one request: latency
        {"name": "attend, 1 token", "op": "attend", "requests": 1, "new": 1, "cached": 4095,
         "page": 16, "e4m3": False, "by_head": False, **stack},
        # a step of a large ragged serving batch over 8-bit pages
        {"name": "attend 8-bit, 64 requests", "op": "attend", "requests": 64, "new": 1,
         "cached": 8191, "page": 64, "e4m3": True, "by_head": True, **stack},
        # a chunk of a long prompt over what was there before, grouped heads
        {"name": "attend, 512 of 32768 tokens", "op": "attend", "requests": 1, "new": 512,
         "cached": 32256, "page": 128, "e4m3": False, "by_head": True, "q_heads": 32,
         "kv_heads": 4, "head_dim": 128},
        # a whole prompt
        {"name": "attend, 8192 tokens", "op": "attend", "requests": 1, "new": 8192, "cached": 0,
         "page": 16, "e4m3": False, "by_head": False, **stack},
        # chunks of all lengths at once, small heads, pages that end inside a tile
        {"name": "attend, 24 chunks", "op": "attend", "requests": 24, "new": 300, "cached": 3000,
         "page": 24, "e4m3": False, "by_head": False, "q_heads": 24, "kv_heads": 8,
         "head_dim": 80},
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo // step, min(hi // step, round(math.exp(
        rng.uniform(math.log(lo / step), math.log(hi / step)))))) * step


_HEADS = [(16, 16), (32, 8), (32, 4), (24, 8), (8, 1), (12, 12)]


def draw(rng):
    op = rng.choice(["rotary", "rotary gradient", "pages", "append", "append", "attend",
                     "attend", "attend"])
    if op.startswith("rotary"):
        dim = rng.choice([64, 80, 96, 128, 128])
        while True:
            c = {"op": op, "tokens": _log_int(rng, 1, 16384), "heads": rng.choice([1, 7, 16, 32, 48]),
                 "head_dim": dim, "part": rng.choice([dim, dim, dim // 2]),
                 "interleaved": rng.random() < 0.5, "factor": rng.choice([1.0, 1.0, 4.0, 16.0])}
            if c["tokens"] * c["heads"] * dim <= 16384 * 32 * 128:
                return c
    page = rng.choice([8, 16, 20, 24, 32, 64, 128, 256])
    if op == "pages":
        while True:
            c = {"op": op, "requests": _log_int(rng, 1, 256), "new": _log_int(rng, 1, 2000),
                 "cached": _log_int(rng, 1, 16384), "page": page, "short": rng.random() < 0.25}
            if _work_tokens(c) <= 8192:
                return c
    heads, kv_heads = rng.choice(_HEADS)
    c = {"op": op, "page": page, "e4m3": rng.random() < 0.4, "by_head": rng.random() < 0.5,
         "q_heads": heads, "kv_heads": kv_heads, "head_dim": rng.choice([64, 80, 96, 128, 128])}
    if op == "append":
        c.update(tokens=_log_int(rng, 1, 8192), interleaved=rng.random() < 0.3,
                 part=rng.choice([c["head_dim"], c["head_dim"] // 2]))
        return c
    while True:
        c.update(requests=_log_int(rng, 1, 128), new=rng.choice([1, 1, _log_int(rng, 1, 4096)]),
                 cached=_log_int(rng, 1, 32768) - 1)
        new, cached = _lengths(c)
        most = max(new) * max(a + b for a, b in zip(new, cached)) * c["requests"]
        keys = (sum(new) + sum(cached)) * kv_heads * c["head_dim"]
        if (most * heads <= 16 * 8192 * 8192 and work(c)["flops"] <= 2.7e11
                and keys <= 64 * 4300 * 16 * 128):
            return c


def _fraction(r, by):
    return 1.0 if r == 0 else (by * r) % 1.0


def _lengths(case):
    """New and cached tokens of each request: the first the most, the others spread."""
    R = case["requests"]
    new = [1 + int((case["new"] - 1) * _fraction(r, 0.7548776662)) for r in range(R)]
    cached = [int(case["cached"] * _fraction(r, 0.6180339887)) for r in range(R)]
    return new, cached


def _work_tokens(case):
    return sum(_lengths(case)[0])


# ------------------------------------------------------------------- inputs

def _frequencies(case):
    """Radians per position of each pair: powers of 10000, slowed down by `factor` where a
    turn takes longer than the original 2048 positions, and between (32 turns in those: as
    they were)."""
    pairs = case["part"] // 2
    f = []
    for i in range(pairs):
        w = 10000.0 ** (-i / pairs)
        turns = 2048 * w / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 31))
        f.append(w * (keep + (1 - keep) / case.get("factor", 1.0)))
    return f


def _turns(case, device):
    """The frequencies in 2^-64 of a turn, modulo 2^64."""
    whole = [round(w / (2 * math.pi) * 2.0 ** 64) for w in _frequencies(case)]
    return torch.tensor([v - (1 << 64) if v >> 63 else v for v in whole], dtype=torch.int64,
                        device=device)


def _positions(T, most, g):
    """Packed sequences of 1000 tokens or less, each from a place of its own."""
    t = torch.arange(T, device="cuda")
    start = torch.randint(0, most, (T // 1000 + 1,), generator=g, device="cuda")
    return (start[t // 1000] + t % 1000).int()


def _by_head(shape, by_head, dtype):
    """An empty cache [pages, page, heads, dim], a head's rows of a page side by side or not."""
    P, S, H, D = shape
    if by_head:
        return torch.empty((P, H, S, D), dtype=dtype, device="cuda").transpose(1, 2)
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)

    op, s = case["op"], {"case": case}
    if op.startswith("rotary"):
        T = case["tokens"]
        s["x"] = normal(T, case["heads"], case["head_dim"])
        s["positions"] = _positions(T, 4096 * int(case["factor"]), g)
        s["turns"] = _turns(case, "cuda")
        # long contexts: scores grow with them, queries and keys each by the root
        s["amplitude"] = 1 + 0.1 * math.log(case["factor"])
        return s
    if op == "pages":
        new, cached = _lengths(case)
        S, R = case["page"], case["requests"]
        have = [-(-c // S) for c in cached]
        want = [-(-(c + n) // S) for c, n in zip(cached, new)]
        fresh = sum(want) - sum(have)
        total = sum(want) + 7
        order = torch.randperm(total, generator=g, device="cuda").int()
        width = max(want) + 2
        used = torch.arange(width, device="cuda") < torch.tensor(have, device="cuda")[:, None]
        s["table"] = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
        s["table"][used] = order[:sum(have)]
        s["pages"] = torch.zeros(total, dtype=torch.int32, device="cuda")
        free = total - sum(have) if not case["short"] else fresh // 2
        s["pages"][:free] = order[sum(have):sum(have) + free]
        s["count"] = torch.tensor([free], dtype=torch.int32, device="cuda")
        s["cached"] = torch.tensor(cached, dtype=torch.int32, device="cuda")
        s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        s["tokens"] = sum(new)
        return s
    S, H, D = case["page"], case["kv_heads"], case["head_dim"]
    if op == "append":
        T = case["tokens"]
        # one projection made all three
        qkv = normal(T, case["q_heads"] + 2 * H, D)
        s["q"], s["k"], s["v"] = qkv.split([case["q_heads"], H, H], 1)
        s["positions"] = _positions(T, 4096, g)
        s["turns"], s["amplitude"] = _turns(case, "cuda"), 1.0
        n_pages = -(-T // S) + 3
        page = torch.randperm(n_pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        s["slots"] = (page[t // S] * S + t % S).int()
    else:
        new, cached = _lengths(case)
        length = [a + b for a, b in zip(new, cached)]
        need = torch.tensor([-(-n // S) for n in length], device="cuda")
        n_pages = int(need.sum()) + 3
        s["table"] = torch.full((case["requests"], int(need.max())), -1, dtype=torch.int32,
                                device="cuda")
        used = torch.arange(int(need.max()), device="cuda") < need[:, None]
        s["table"][used] = torch.randperm(n_pages, generator=g, device="cuda")[:-3].int()
        offsets = [0]
        for n in new:
            offsets.append(offsets[-1] + n)
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        s["context"] = torch.tensor(length, dtype=torch.int32, device="cuda")
        s["longest"], s["most"] = max(new), max(length)
        s["q"] = normal(offsets[-1], case["q_heads"], D, scale=2.0)
    for name in ("key", "value"):
        c = _by_head((n_pages, S, H, D), case["by_head"], E4M3 if case["e4m3"] else BF16)
        x = torch.randn(c.shape, generator=g, device="cuda")
        if case["e4m3"]:
            c.copy_(x.mul_(64).to(E4M3))
            e = torch.empty((n_pages, H, S), dtype=torch.uint8, device="cuda")
            s[name + "_exponent"] = e.random_(BIAS - 7, BIAS - 5, generator=g).transpose(1, 2)
        else:
            c.copy_(x)
            s[name + "_exponent"] = None
        s[name] = c
    return s


# -------------------------------------------------------------- plain forms

def _rotated(x, positions, turns, amplitude, interleaved, sign=1):
    """x [tokens, heads, dim] in 32 bits; angles in whole 2^-64 of a turn, so that far
    positions lose nothing, then in 64 bits."""
    pairs = turns.numel()
    angle = (positions.long()[:, None] * turns).double() * (2 * math.pi * 2.0 ** -64)
    cos = (torch.cos(angle) * amplitude).float()[:, None]
    sin = (torch.sin(angle) * (sign * amplitude)).float()[:, None]
    if interleaved:
        a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
    else:
        a, b = x[..., :pairs], x[..., pairs:2 * pairs]
    y = a * cos - b * sin, a * sin + b * cos
    y = torch.stack(y, 3).flatten(2) if interleaved else torch.cat(y, 2)
    return torch.cat([y, x[..., 2 * pairs:]], 2)


def _exponents(most):
    """Of e4m3 rows: the least e with most <= 448 * 2^e."""
    m, e = torch.frexp(most)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(most > 0, e, LOWEST).clamp(LOWEST, HIGHEST)
    return torch.where(torch.isfinite(most), e, 128)


def _to_e4m3(y, e):
    return torch.ldexp(y, -e[..., None]).clamp(-448, 448).to(E4M3)


def _pairs_most(x, turns, amplitude, interleaved):
    """A bound of a rotated row's values, the same however cos and sin are computed: the
    largest |a| + |b| of a pair, or |x| behind the pairs."""
    pairs = turns.numel()
    if interleaved:
        a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
    else:
        a, b = x[..., :pairs], x[..., pairs:2 * pairs]
    most = (a.abs() + b.abs()).amax(2) * amplitude
    rest = x[..., 2 * pairs:]
    return torch.maximum(most, rest.abs().amax(2)) if rest.shape[2] else most


def _values(cache, exponent):
    return cache.float() if exponent is None else torch.ldexp(cache.float(),
                                                              exponent.int()[..., None] - BIAS)


def _pages(s):
    S, T = s["case"]["page"], s["tokens"]
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    width = table.shape[1]
    have, want = (cached + S - 1) // S, (cached + new + S - 1) // S
    take = want - have
    total = take.cumsum(0)
    granted = (take == 0) | (total <= s["count"])
    column = torch.arange(width, device=table.device)
    fresh = (column >= have[:, None]) & (column < want[:, None]) & granted[:, None]
    rank = (total - take - have)[:, None] + column
    at = (s["count"] - 1 - rank).clamp(0, s["pages"].numel() - 1)
    table = torch.where(fresh, s["pages"][at], table)
    offsets = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    t = torch.arange(T, device=table.device)
    r = torch.searchsorted(offsets[1:], t, right=True)
    position = cached[r] + t - offsets[r]
    slot = table[r, (position // S).clamp(max=width - 1)] * S + position % S
    return {"table": table, "offsets": offsets.int(),
            "context": torch.where(granted, cached + new, 0).int(),
            "lengths": torch.where(granted, cached + new, cached).int(),
            "positions": position.int(), "slots": torch.where(granted[r], slot, -1).int(),
            "count": s["count"] - torch.where(granted, take, 0).sum().int()}


def _append(s):
    case = s["case"]
    turn = s["turns"], s["amplitude"], case["interleaved"]
    slots = s["slots"].long()
    page, at = slots // case["page"], slots % case["page"]
    k, v = s["k"].float(), s["v"].float()
    out = {"q": _rotated(s["q"].float(), s["positions"], *turn).to(BF16)}
    rows = {"key": _rotated(k, s["positions"], *turn), "value": v}
    if case["e4m3"]:
        most = {"key": _pairs_most(k, *turn), "value": v.abs().amax(2)}
        e = {n: _exponents(m) for n, m in most.items()}
        rows = {n: _to_e4m3(y, e[n]) for n, y in rows.items()}
        out["key_exponent"] = s["key_exponent"].index_put_((page, at), (e["key"] + BIAS).byte())
        out["value_exponent"] = s["value_exponent"].index_put_((page, at),
                                                               (e["value"] + BIAS).byte())
    out["key"] = _put(s["key"], page, at, rows["key"])
    out["value"] = _put(s["value"], page, at, rows["value"])
    return out


def _put(cache, page, at, rows):
    if cache.dtype is E4M3:
        cache.view(torch.uint8).index_put_((page, at), rows.view(torch.uint8))
        return cache
    return cache.index_put_((page, at), rows.to(BF16))


def _attend(s):
    """Padded to the longest request: [requests, heads, new tokens, keys]."""
    case = s["case"]
    R, N, L = case["requests"], s["longest"], s["most"]
    Hq, H, D, S = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    offsets, context, table = s["offsets"].long(), s["context"].long(), s["table"].long()
    device = table.device
    new = offsets[1:] - offsets[:-1]
    key, i = torch.arange(L, device=device), torch.arange(N, device=device)
    page = table[:, key // S].clamp(min=0)                       # [R, L]
    there = (key < context[:, None])[:, :, None, None]

    def rows(name):
        e = s[name + "_exponent"]
        x = _values(s[name][page, key % S], None if e is None else e[page, key % S])
        return torch.where(there, x, 0.0).transpose(1, 2)        # [R, H, L, D]

    live = i < new[:, None]
    token = (offsets[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][token].float().view(R, N, H, Hq // H, D).permute(0, 2, 3, 1, 4)
    score = (q.reshape(R, H, -1, D) @ rows("key").transpose(2, 3)).view(R, H, -1, N, L)
    score = score * D ** -0.5
    seen = key <= (context - new)[:, None, None] + i[:, None]     # [R, N, L]
    score = torch.where(seen[:, None, None], score, -math.inf)
    p = torch.exp(score - score.amax(4, keepdim=True))
    p = p / p.sum(4, keepdim=True)
    o = (p.view(R, H, -1, L) @ rows("value")).view(R, H, -1, N, D)
    o = o.permute(0, 3, 1, 2, 4).reshape(R, N, Hq, D).to(BF16)
    return o[live]


# ------------------------------------------------------------------ one pass

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        if op.startswith("rotary"):
            return _rotated(s["x"].float(), s["positions"], s["turns"], s["amplitude"],
                            case["interleaved"], -1 if op == "rotary gradient" else 1).to(BF16)
        return {"pages": _pages, "append": _append, "attend": _attend}[op](s)
    from lossless_exponent_reuse_gb300 import attention
    if op.startswith("rotary"):
        rotary = attention.Rotary(s["turns"], s["amplitude"], case["interleaved"])
        call = attention.rotary if op == "rotary" else attention.rotary_backward
        return call(s["x"], s["positions"], rotary)
    if op == "pages":
        pool = attention.Pool(s["table"], s["pages"], s["count"])
        r = attention.assign_pages(pool, s["cached"], s["new"], s["tokens"], case["page"])
        return {"table": r.pool.table, "offsets": r.offsets, "context": r.context,
                "lengths": r.lengths, "positions": r.positions, "slots": r.slots,
                "count": r.pool.count}
    cache = attention.Cache(s["key"], s["value"], s["key_exponent"], s["value_exponent"])
    if op == "append":
        rotary = attention.Rotary(s["turns"], s["amplitude"], case["interleaved"])
        out = {"q": attention.append(s["q"], s["k"], s["v"], s["positions"], s["slots"], rotary,
                                     cache),
               "key": cache.key, "value": cache.value}
        if case["e4m3"]:
            out.update(key_exponent=cache.key_exponent, value_exponent=cache.value_exponent)
        return out
    return attention.attend(s["q"], cache, s["table"], s["offsets"], s["context"],
                            longest=s["longest"])


def work(case):
    op = case["op"]
    if op.startswith("rotary"):
        rows = case["tokens"] * case["heads"]
        return {"bytes": 4 * rows * case["head_dim"] + 4 * case["tokens"] + 4 * case["part"],
                "flops": 3 * rows * case["part"]}
    if op == "pages":
        # lengths in; offsets, contexts and lengths out; a position and a slot per token; the
        # free pages taken and their places in the table; the page that each request had begun
        new, cached = _lengths(case)
        S, R = case["page"], case["requests"]
        fresh = sum(-(-(c + n) // S) + -c // S for c, n in zip(cached, new))
        return {"bytes": 24 * R + 8 * sum(new) + 8 * fresh, "flops": 4 * sum(new)}
    Hq, H, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    size = 1 + 1 / D if case["e4m3"] else 2
    if op == "append":
        T = case["tokens"]
        return {"bytes": int(T * D * (4 * Hq + 4 * H + 2 * size * H) + 8 * T + 4 * case["part"]),
                "flops": 3 * T * (Hq + H) * case["part"]}
    new, cached = _lengths(case)
    seen = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, cached))
    keys = sum(new) + sum(cached)
    return {"bytes": int(4 * sum(new) * Hq * D + 2 * keys * H * D * size + 4 * keys / case["page"]),
            "flops": 4 * seen * Hq * D}


# ------------------------------------------------------- definitions, 64 bits

def _turned(x, case, positions, amplitude, sign):
    """Each pair (a, b) as the complex number a + i b, times amplitude * exp(i angle)."""
    w = torch.tensor(_frequencies(case), dtype=torch.float64, device=x.device)
    n = w.numel()
    at = torch.arange(n, device=x.device)
    first, second = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + n)
    angle = sign * positions.double()[:, None] * w
    z = torch.complex(x[..., first], x[..., second])
    z = z * torch.polar(torch.full_like(angle, amplitude), angle)[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None                # whole numbers alone
    s = prepare(case, seed)
    if op.startswith("rotary"):
        return _turned(s["x"].double(), case, s["positions"], s["amplitude"],
                       1 if op == "rotary" else -1)
    if op == "append":
        k, v, slots = s["k"].double(), s["v"].double(), s["slots"].long()
        page, at = slots // case["page"], slots % case["page"]
        out = {"q": _turned(s["q"].double(), case, s["positions"], s["amplitude"], 1)}
        new = {"key": _turned(k, case, s["positions"], s["amplitude"], 1), "value": v}
        for name, y in new.items():
            if case["e4m3"]:
                # y / 2^e with the power of two that the row is stored with: the least that
                # leaves room for every |a| + |b| of a rotated pair, or |x|
                n = case["part"] // 2 if name == "key" else 0
                i = torch.arange(n, device=y.device)
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + n)
                x = k if name == "key" else v
                most = x[..., 2 * n:].abs()
                if n:
                    pair = (x[..., a].abs() + x[..., b].abs()) * s["amplitude"]
                    most = torch.cat([most, pair], 2)
                e = torch.ceil(torch.log2(most.amax(2) / 448)).clamp(LOWEST, HIGHEST)
                y = y * torch.exp2(-e)[..., None]
                out[name + "_exponent"] = None
            cache = s[name].double()
            cache[page, at] = y
            out[name] = cache
        return out
    Hq, H, D, S = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    new, cached = _lengths(case)
    if 4 * Hq * D * sum(n * (n + c) for n, c in zip(new, cached)) > 4e12:
        return None
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for r, (n, c) in enumerate(zip(new, cached)):
        at = torch.arange(n + c, device="cuda")
        page = s["table"][r].long()[at // S]
        rows = {}
        for name in ("key", "value"):
            x = s[name][page, at % S].double()
            if case["e4m3"]:
                x = x * 2.0 ** (s[name + "_exponent"][page, at % S].double() - BIAS)[..., None]
            rows[name] = x
        hidden = at > c + torch.arange(n, device="cuda")[:, None]
        for h in range(Hq):
            score = s["q"][row:row + n, h].double() @ rows["key"][:, h * H // Hq].T
            score = (score / math.sqrt(D)).masked_fill(hidden, -math.inf)
            p = torch.softmax(score, 1)
            o[row:row + n, h] = p @ rows["value"][:, h * H // Hq]
        row += n
    return o
