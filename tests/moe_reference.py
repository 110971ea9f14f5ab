"""The mixture-of-experts operators in 64 bits, written from their formulas
with loops and torch's elementary operations; and what their outputs may be
off.

Bounds.  An output rounded once to bf16 (8 significant bits) is within
2^-8 of its value, relative; to e4m3 (4 significant bits) within 2^-4, or
half a step of its smallest values, 2^-10, times the scale.  A 32-bit sum of
K terms a_i b_i in any order, each operation within 2^-23 (truncation
allowed), is within (K + 2) 2^-23 sum|a_i b_i| of the exact one: `slack`
tensors below hold the sum of the terms' magnitudes.
"""
import math

import torch

U_BF16 = 2.0 ** -8
U_F32 = 2.0 ** -23
E4M3_MAX = 448.0
TINY = 1e-30


def within(got, want, slack, what="", rounded=U_BF16):
    """got is `rounded`-close to some value within slack of want."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    limit = rounded * (want.abs() + slack) + slack + 1e-38
    off = (got - want).abs() - limit
    assert torch.isfinite(got).all() or not torch.isfinite(want).all(), what
    bad = off > 0
    assert not bad.any(), (what, int(bad.sum()), float(off.max()),
                           float((got - want).abs().max()))


def norm(x, weight, residual, eps):
    s = x.double() + (0 if residual is None else residual.double())
    rstd = ((s * s).mean(1) + eps) ** -0.5
    return s, rstd, s * rstd[:, None] * weight.double()


def quantize(y):
    """scale and y / scale, not rounded."""
    scale = y.abs().amax(-1).clamp(min=TINY) / E4M3_MAX
    return scale, y / scale[..., None]


def route(logits, k, mask=None):
    """experts [T, k], softmax weights [T, k] and the order, by plain loops."""
    T, E = logits.shape
    rows = logits.double().tolist()
    live = [True] * T if mask is None else [bool(m) for m in mask.tolist()]
    experts, weights = [], []
    for t in range(T):
        l = rows[t]
        order = sorted(range(E), key=lambda e: (-math.inf if l[e] != l[e] else -l[e], e))
        pick = [e for e in order[:k] if l[e] != l[e] or l[e] > -math.inf] if live[t] else []
        top = max((v for v in l if v == v), default=0.0)
        z = sum(math.exp(v - top) for v in l) if top > -math.inf else 1.0
        experts.append(pick + [-1] * (k - len(pick)))
        weights.append([math.exp(l[e] - top) / z for e in pick] + [0.0] * (k - len(pick)))
    pairs = sorted((experts[t][j], t, j) for t in range(T) for j in range(k)
                   if experts[t][j] >= 0)
    slots = [[-1] * k for _ in range(T)]
    tokens = [-1] * (T * k)
    offsets = [0] * (E + 1)
    for at, (e, t, j) in enumerate(pairs):
        slots[t][j] = at
        tokens[at] = t
        offsets[e + 1] += 1
    for e in range(E):
        offsets[e + 1] += offsets[e]
    return experts, weights, slots, tokens, offsets


def bounds(offsets, rows):
    """The groups as the calls read them: clamped and non-decreasing."""
    at, out = 0, []
    for v in offsets.tolist()[1:]:
        to = min(max(v, at), rows)
        out.append((at, to))
        at = to
    return out


def gather(x, tokens, rows):
    if tokens is None:
        return x.double()[:rows]
    t = tokens.long()
    ok = (t >= 0) & (t < x.shape[0])
    return torch.where(ok[:, None], x.double()[t.clamp(0, x.shape[0] - 1)], 0.0)


def product(rows, w, offsets):
    """rows [R, K] times w [E, N, K], and the sums of the terms' magnitudes."""
    R, N = rows.shape[0], w.shape[1]
    y = torch.zeros(R, N, dtype=torch.float64, device=rows.device)
    size = torch.zeros_like(y)
    for e, (a, b) in enumerate(bounds(offsets, R)):
        we = w[e].double()
        y[a:b] = rows[a:b] @ we.T
        size[a:b] = rows[a:b].abs() @ we.abs().T
    return y, size


def product_dw(dy, x, offsets, N, K):
    E = offsets.numel() - 1
    out = torch.zeros(E, N, K, dtype=torch.float64, device=dy.device)
    size = torch.zeros_like(out)
    for e, (a, b) in enumerate(bounds(offsets, dy.shape[0])):
        out[e] = dy[a:b].double().T @ x[a:b]
        size[e] = dy[a:b].double().abs().T @ x[a:b].abs()
    return out, size


def silu(g):
    return g / (1 + torch.exp(-g))


def gated(pre):
    g, u = pre.chunk(2, 1)
    return silu(g) * u


def gated_gradient(d, pre):
    g, u = pre.chunk(2, 1)
    s = 1 / (1 + torch.exp(-g))
    return torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], 1)
