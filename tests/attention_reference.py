"""The attention half's operators in 64 bits, written from their formulas with
loops and torch's elementary operations, inputs for their tests, and what their
outputs may be off.

Bounds, beside moe_reference's.

rotary: the angle is a multiple of 2^-24 of a half turn (2^-23.3 rad off at
most), sine and cosine within 2 units of 2^-24, the amplitude, two products and
a sum each within 2^-24: less than 2^-21 (|a| + |b|) s together.

attend: a score is off by (D + 4) 2^-23 sum|q k| scale, which moves a weight by
as much, relative, and their sum too; a weight is rounded to 8 bits (2^-8); the
weights' exponential and the 32-bit sums add (L + 64) 2^-22.  With A = sum p|v|:
A (2^-8 + 4 ds + (L + 64) 2^-22).  A single weight's rounding is as often up as
down, so that over many values the 2-norm is off by less: the weights' part and
the output's are both 2^-8 / sqrt(3) at most, 2^-8 sqrt(2/3) together.
"""
import math

import torch

from lossless_exponent_reuse_gb300 import attention
from moe_reference import within

BF16, F32, E4M3, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


def rand(*shape, seed=0, scale=1.0, dtype=BF16, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=device) * scale).to(dtype)


def ints(v, device="cuda"):
    return torch.tensor(v, dtype=I32, device=device)


def pair_places(pairs, interleaved):
    return [(2 * i, 2 * i + 1) if interleaved else (i, i + pairs) for i in range(pairs)]


def angles(positions, turns):
    """Of whole numbers, then of fractions: [tokens, pairs]."""
    rows = [[((p * t) % (1 << 64)) / 2.0 ** 64 for t in turns.tolist()]
            for p in positions.tolist()]
    return torch.tensor(rows, dtype=torch.float64).reshape(len(rows), turns.numel()) * 2 * math.pi


def rotary(x, positions, r, sign=1):
    """y, and the slack of each value."""
    x = x.double().cpu()
    y, slack = x.clone(), torch.zeros_like(x)
    t = sign * angles(positions, r.turns)[:, None]
    cos, sin = torch.cos(t) * r.amplitude, torch.sin(t) * r.amplitude
    for i, (a, b) in enumerate(pair_places(r.turns.numel(), r.interleaved)):
        y[..., a] = x[..., a] * cos[..., i] - x[..., b] * sin[..., i]
        y[..., b] = x[..., a] * sin[..., i] + x[..., b] * cos[..., i]
        slack[..., a] = slack[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(r.amplitude)
    return y, slack * 2.0 ** -21


def exponents(x, r=None):
    """Of e4m3 rows, biased: of values, or of rows to be rotated by r."""
    x = x.double().cpu()
    m = x.abs()
    if r is not None:
        for a, b in pair_places(r.turns.numel(), r.interleaved):
            m[..., a] = m[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(r.amplitude)
    m = m.amax(-1)
    e = torch.ceil(torch.log2(m / 448)).clamp(-100, 119) + 127
    return torch.where(torch.isfinite(m), e, 255.0).to(torch.uint8)


def values(cache, exponent):
    """The cache in 64 bits."""
    v = cache.double()
    if exponent is None:
        return v
    scale = torch.exp2(exponent.double() - 127)
    return v * torch.where(exponent == 255, math.nan, scale)[..., None]


def assign(table, free, count, cached, new, tokens, page):
    """By plain loops; table is changed."""
    offsets, context, lengths, positions, slots = [0], [], [], [], []
    out, at, starved = count, 0, False
    width = len(table[0]) if table else 0
    for r, (c, n) in enumerate(zip(cached, new)):
        c, n = max(c, 0), max(n, 0)
        held, want = -(-c // page), -(-(c + n) // page)
        fits = at + n <= tokens and want <= width and c + n < 2 ** 31
        if not fits or (want > held and (starved or want - held > out)):
            starved = True
            granted = False
        else:
            granted = True
            for i in range(held, want):
                out -= 1
                table[r][i] = free[out]
        for i in range(n):
            if len(slots) == tokens:
                break
            p = c + i
            positions.append((p + 2 ** 31) % 2 ** 32 - 2 ** 31)   # 32 bits
            slots.append(table[r][p // page] * page + p % page if granted else -1)
        at += n
        offsets.append(min(at, tokens))
        context.append(c + n if granted else 0)
        lengths.append(c + n if granted else c)
    positions += [0] * (tokens - len(positions))
    slots += [-1] * (tokens - len(slots))
    return offsets, context, lengths, positions, slots, out


def paged(lengths, page, heads, dim, seed=0, e4m3=False, by_head=False, extra=2, value=None):
    """A cache that holds requests of these lengths, and their table; every place
    that holds no key is NaN.  ``value(kind, request, n)``: rows [n, heads, dim] if not
    random."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + extra
    g = torch.Generator(device="cuda").manual_seed(seed)
    order = torch.randperm(pages, generator=g, device="cuda").tolist()
    width = max(need + [1]) + 1
    table, rows = torch.full((len(lengths), width), -1, dtype=I32), []
    for r, n in enumerate(need):
        rows.append([order.pop() for _ in range(n)])
        table[r, :n] = ints(rows[r], "cpu")
    table = table.cuda()
    sides, marks = [], []
    for kind in (0, 1):
        shape = (pages, heads, page, dim) if by_head else (pages, page, heads, dim)
        c = torch.full(shape, math.nan, device="cuda").to(E4M3 if e4m3 else BF16)
        c = c.transpose(1, 2) if by_head else c
        e = torch.full((pages, heads, page), 255, dtype=torch.uint8, device="cuda").transpose(1, 2)
        for r, n in enumerate(lengths):
            x = (rand(n, heads, dim, seed=seed * 1000 + 2 * r + kind, dtype=F32) if value is None
                 else value(kind, r, n))
            at = torch.arange(n, device="cuda")
            slot = (torch.tensor(rows[r] + [0], device="cuda")[at // page], at % page)
            if e4m3:
                k = rand(n, heads, seed=seed * 1000 + 2 * r + kind + 500, dtype=F32)
                k = k.mul(2).round().clamp(-6, 6)        # rows of several magnitudes
                e[slot] = (k + 127 - 6).to(torch.uint8)
                x = (x * 64).clamp(-448, 448)
                c.view(torch.uint8)[slot] = x.to(E4M3).view(torch.uint8)
            else:
                c[slot] = x.to(BF16)
        sides.append(c)
        marks.append(e if e4m3 else None)
    return attention.Cache(*sides, *marks), table


def attend(q, cache, table, offsets, context, scale=None):
    """o and its slack, by a loop over requests and heads."""
    T, Hq, D = q.shape
    P, S, H, _ = cache.key.shape
    scale = D ** -0.5 if scale is None else scale
    o = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    slack = torch.zeros_like(o)
    off = [0] + [min(max(v, 0), T) for v in offsets.tolist()[1:]]
    for r, L in enumerate(context.tolist()):
        a, b = off[r], off[r + 1]
        L = min(max(L, 0), table.shape[1] * S)
        if b <= a or L == 0:
            continue
        at = torch.arange(L, device=q.device)
        page = table[r].long()[at // S]
        there = (page >= 0) & (page < P)
        slot = page.clamp(0, P - 1), at % S
        K, V = (torch.where(there[:, None, None],
                            values(x.view(torch.uint8)[slot].view(x.dtype) if e is not None
                                   else x[slot], None if e is None else e[slot]), 0.0)
                for x, e in ((cache.key, cache.key_exponent), (cache.value, cache.value_exponent)))
        seen = at < L - (b - a) + torch.arange(b - a, device=q.device)[:, None] + 1
        live = seen.any(1)
        hidden = ~seen[live]
        for h in range(Hq):
            k, v = K[:, h * H // Hq], V[:, h * H // Hq]
            qh = q[a:b, h].double()
            s = torch.where(seen, (qh @ k.T) * scale, -math.inf)
            p = torch.softmax(s[live], 1)
            size = torch.where(seen, qh.abs() @ torch.nan_to_num(k.abs(), 0, 0, 0).T, 0.0)
            ds = (D + 4) * 2.0 ** -23 * abs(scale) * size.amax(1, keepdim=True)
            # keys that are not seen have no part, whatever they hold
            clean = torch.nan_to_num(v, 0, 0, 0)
            out, A = p @ clean, p @ clean.abs()
            for j in (v != clean).any(1).nonzero()[:, 0].tolist():
                out = out + torch.where(hidden[:, j, None], 0.0, p[:, j, None] * (v[j] - clean[j]))
            rows = torch.zeros(b - a, D, dtype=torch.float64, device=q.device)
            size = torch.zeros_like(rows)
            rows[live], size[live] = out, A
            o[a:b, h] = rows
            slack[a:b, h] = size * (2.0 ** -8 + 4 * ds + (L + 64) * 2.0 ** -22)
    return o, slack


def check_attend(got, q, cache, table, offsets, context, scale=None, what=""):
    want, slack = attend(q, cache, table, offsets, context, scale)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    got = got.double()
    odd = ~fine & ~torch.isnan(want)
    assert torch.equal(got[odd], want[odd]), what
    got, want, slack = (torch.where(fine, x, 0.0) for x in (got, want, slack))
    within(got, want, slack, what)
    if want.numel() >= 4096:
        assert (got - want).norm() <= 2.0 ** -8 * want.norm(), what
