"""The operators of a mixture-of-experts layer next to the Allgather that
rebuilds its weights: sizes to measure them at, their plain forms, and their
definitions in 64 bits.

Four operators, each with its gradient where training needs one:

  norm     root-mean-square norm of x + residual, scaled by a weight; the sum
           is kept for the next residual.  Output in bf16, or in e4m3 with one
           scale per row.
  route    choice of k experts per token from router logits (softmax over all
           experts, ties to the lowest index), and the order that groups the
           (token, expert) pairs by expert.
  combine  a token's output from the rows its experts made, weighted.
  experts  matrix products grouped by expert, with ragged group sizes: gate
           and up with the gated unit silu(gate) * up, and down.  The weights
           are views of the flat bucket that the Allgather rebuilds (for each
           expert gate, up, down), or e4m3 with one scale per output feature.

Sizes: OLMoE's layer (64 experts of 2048 x 1024, 8 chosen) and the
fine-grained layer (128 experts of 1536 x 4096), the framework's own
workloads, from one token to a training batch, and odd sizes around them.
"""
import math

import torch

own = False

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6
E4M3_MAX = 448.0
TINY = 1e-30          # an all-zero row's amax is raised to this, so that its scale is not 0


# ---------------------------------------------------------------- the cases

def listed():
    olmoe = {"experts": 64, "dim": 2048, "ff": 1024, "topk": 8}
    fine = {"experts": 128, "dim": 1536, "ff": 4096, "topk": 8}
    return [
        # one token of a serving step before 8-bit expert products: latency
        {"name": "norm 8-bit, 1 token", "op": "norm", "tokens": 1, "dim": 2048, "quantize": True},
        # a training batch's activations (8 sequences of 2048), bf16
        {"name": "norm, 16384 tokens", "op": "norm", "tokens": 16384, "dim": 2048,
         "quantize": False},
        # the gradient of a ragged batch of the fine-grained layer
        {"name": "norm gradient, 10007 tokens", "op": "norm gradient", "tokens": 10007,
         "dim": 1536},
        # one token of a serving step: latency
        {"name": "route, 1 token", "op": "route", "tokens": 1, "experts": 64, "topk": 8,
         "logits": "f32", "renormalize": False, "masked": 0.0},
        # a training batch over the fine-grained layer's experts, with padding tokens
        {"name": "route, 16384 tokens", "op": "route", "tokens": 16384, "experts": 128,
         "topk": 8, "logits": "bf16", "renormalize": True, "masked": 0.05},
        # a serving batch's rows back to its tokens
        {"name": "combine, 333 tokens", "op": "combine", "tokens": 333, "masked": 0.0, **olmoe},
        # the gradients of a training batch's combination and of its router's logits
        {"name": "combine gradient, 8192 tokens", "op": "combine gradient", "tokens": 8192,
         "masked": 0.05, **olmoe},
        # one token of a serving step: 8 rows, each its own expert's weights
        {"name": "experts, 1 token", "op": "experts", "tokens": 1, "train": False, "masked": 0.0,
         **olmoe},
        # a small serving batch over the fine-grained layer's 8-bit weights
        {"name": "experts 8-bit, 24 tokens", "op": "experts 8-bit", "tokens": 24, "masked": 0.0,
         **fine},
        # a prompt through 8-bit weights
        {"name": "experts 8-bit, 4096 tokens", "op": "experts 8-bit", "tokens": 4096,
         "masked": 0.0, **olmoe},
        # a training batch's forward pass, what the gradient needs kept, padding tokens
        {"name": "experts, 8192 tokens", "op": "experts", "tokens": 8192, "train": True,
         "masked": 0.02, **olmoe},
        # and its gradients of inputs and weights
        {"name": "experts gradient, 8192 tokens", "op": "experts gradient", "tokens": 8192,
         "masked": 0.02, **olmoe},
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo // step, min(hi // step, round(math.exp(
        rng.uniform(math.log(lo / step), math.log(hi / step)))))) * step


def draw(rng):
    kind = rng.choice(["norm", "norm gradient", "route", "combine", "combine gradient",
                       "experts", "experts 8-bit", "experts gradient"])
    masked = rng.choice([0.0, 0.0, rng.uniform(0.01, 0.3)])
    c = {"op": kind, "tokens": _log_int(rng, 1, 16384)}
    if kind == "norm":
        return {**c, "dim": _log_int(rng, 64, 3000), "quantize": rng.random() < 0.5}
    if kind == "norm gradient":
        return {**c, "dim": _log_int(rng, 64, 1500)}
    if kind == "route":
        c.update(experts=rng.choice([8, 16, 60, 64, 100, 128]), topk=rng.choice([1, 2, 4, 6, 8]),
                 logits=rng.choice(["f32", "bf16"]), renormalize=rng.random() < 0.5,
                 masked=masked)
        return c
    c.update(experts=rng.choice([8, 16, 60, 64, 128]), topk=rng.choice([1, 2, 4, 6, 8]),
             masked=masked)
    if kind.startswith("combine"):
        c["tokens"] = _log_int(rng, 1, 8192)
        c["dim"] = _log_int(rng, 128, 2048, 8)
        return c
    step = 16 if kind == "experts 8-bit" else 8
    while True:
        c.update(tokens=_log_int(rng, 1, 8192), dim=_log_int(rng, 256, 3000, step),
                 ff=_log_int(rng, 128, 3000, step))
        if kind == "experts":
            c["train"] = rng.random() < 0.5
        cost = c["tokens"] * c["topk"] * c["dim"] * c["ff"]
        room = c["experts"] * c["dim"] * c["ff"]
        if cost <= 8192 * 8 * 2048 * 1024 and room <= 128 * 1536 * 4096:
            return c


# ------------------------------------------------------------------- inputs

def _routing(logits, k, live):
    """Experts, weights and the order of the pairs by expert (int64 and f32)."""
    T, E = logits.shape
    l = logits.float()
    value, index = torch.sort(l, dim=1, descending=True, stable=True)
    value, index = value[:, :k], index[:, :k]
    p = torch.exp(l - l.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    chosen = (value > -math.inf) & live[:, None]
    weights = torch.where(chosen, p.gather(1, index), 0.0)
    experts = torch.where(chosen, index, -1)
    return weights, experts, _order(experts, E)


def _order(experts, E):
    """slots [T, k], tokens [T k] and offsets [E + 1] of a choice of experts."""
    T, k = experts.shape
    group = torch.where(experts < 0, E, experts).reshape(-1)
    by, order = torch.sort(group, stable=True)
    offsets = torch.searchsorted(by, torch.arange(E + 1, device=by.device))
    place = torch.arange(T * k, device=by.device)
    slots = torch.empty_like(place)
    slots[order] = place
    slots = torch.where(group < E, slots, -1).reshape(T, k)
    tokens = torch.where(place < offsets[E], order // k, -1)
    return slots, tokens, offsets


def _bucket(case, g):
    """The rebuilt bucket of bf16 weights and its views: gate and up, down."""
    E, D, F = case["experts"], case["dim"], case["ff"]
    b = torch.empty(E * 3 * F * D, dtype=BF16, device="cuda").normal_(0, 0.02, generator=g)
    return (b.as_strided((E, 2 * F, D), (3 * F * D, D, 1)),
            b.as_strided((E, D, F), (3 * F * D, F, 1), 2 * F * D))


def _rows_to_e4m3(x):
    scale = x.float().abs().amax(-1).clamp(min=TINY) / E4M3_MAX
    return (x.float() / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, T = case["op"], case["tokens"]

    def normal(*shape, scale=1.0, dtype=BF16):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if op.startswith("norm"):
        D = case["dim"]
        s["weight"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(BF16)
        if op == "norm":
            s["x"], s["residual"] = normal(T, D), normal(T, D, scale=3.0)
        else:
            s["dy"], s["dh"] = normal(T, D, scale=0.01), normal(T, D, scale=0.01)
            s["h"] = normal(T, D, scale=3.0)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        return s

    # router logits with favoured experts, so that the groups are ragged
    E, k = case["experts"], case["topk"]
    logits = (torch.randn((T, E), generator=g, device="cuda")
              + 0.5 * torch.randn(E, generator=g, device="cuda"))
    logits = logits.to(F32 if case.get("logits", "f32") == "f32" else BF16)
    live = torch.rand(T, generator=g, device="cuda") >= case["masked"]
    if op == "route":
        s["logits"], s["live"] = logits, live if case["masked"] else None
        return s
    weights, experts, (slots, tokens, offsets) = _routing(logits, k, live)
    s["slots"], s["tokens"], s["offsets"] = slots.int(), tokens.int(), offsets.int()
    if op.startswith("combine"):
        s["weights"] = weights
        s["rows"] = normal(T * k, case["dim"])
        if op == "combine gradient":
            s["logits"], s["experts"] = logits, experts.int()
            s["dy"] = normal(T, case["dim"], scale=0.01)
        return s

    # for the plain form alone: the longest group (the kernels read the offsets on the device)
    s["longest"] = int((offsets[1:] - offsets[:-1]).max())
    D, F, R = case["dim"], case["ff"], T * k
    gate_up, down = _bucket(case, g)
    if op == "experts 8-bit":
        s["x"], s["x_scale"] = _rows_to_e4m3(normal(T, D))
        s["gate_up"], s["gate_up_scale"] = _rows_to_e4m3(gate_up)
        s["down"], s["down_scale"] = _rows_to_e4m3(down)
        return s
    s["gate_up"], s["down"] = gate_up, down
    s["x"] = normal(T, D)
    if op == "experts gradient":
        s["dy"] = normal(R, D, scale=0.01)
        s["pre"] = normal(R, 2 * F, scale=0.02 * math.sqrt(D))
        gate, up = s["pre"].float().split(F, 1)
        s["h"] = (gate * torch.sigmoid(gate) * up).to(BF16)
    return s


# -------------------------------------------------------------- plain forms

def _groups(s):
    """Group of each row, its place in it, and whether the row is in use."""
    offsets, E = s["offsets"].long(), s["case"]["experts"]
    row = torch.arange(s["tokens"].numel(), device=offsets.device)
    group = torch.searchsorted(offsets, row, right=True) - 1
    live = row < offsets[E]
    group = torch.where(live, group, 0)
    return group, torch.where(live, row - offsets[group], 0), live


def _gathered(x, tokens):
    return x.float()[tokens.long().clamp(min=0)] * (tokens >= 0)[:, None]


def _pad(rows, s, groups):
    """[E, longest, n] from rows in expert order, zeros beyond each group."""
    group, place, live = groups
    E, longest = s["case"]["experts"], max(s["longest"], 1)
    out = torch.zeros((E * longest + 1, rows.shape[1]), device=rows.device)
    out[torch.where(live, group * longest + place, E * longest)] = rows
    return out[:-1].view(E, longest, -1)


def _unpad(padded, groups):
    group, place, live = groups
    return torch.where(live[:, None], padded[group, place], 0.0)


def _product(rows, w, s, groups):
    """rows [R, K] in expert order times w [E, N, K], each with its group's."""
    group, _, live = groups
    if rows.shape[0] < w.shape[0]:     # fewer rows than experts: only their weights
        y = torch.bmm(w[group].float(), rows[:, :, None])[:, :, 0]
        return torch.where(live[:, None], y, 0.0)
    return _unpad(torch.bmm(_pad(rows, s, groups), w.float().transpose(1, 2)), groups)


def _product_dw(dy, x, s, groups):
    return torch.bmm(_pad(dy, s, groups).transpose(1, 2), _pad(x, s, groups))


def _gated(pre):
    gate, up = pre.chunk(2, 1)
    return gate * torch.sigmoid(gate) * up


def _gated_gradient(dh, pre):
    gate, up = pre.chunk(2, 1)
    sig = torch.sigmoid(gate)
    return torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], 1)


def _route_gradient(dweights, weights, experts, logits, renormalize):
    """Of the logits, from the gradient of the chosen experts' weights."""
    inner = (dweights * weights).sum(1, keepdim=True)
    chosen = experts >= 0
    index = experts.long().clamp(min=0)
    if renormalize:
        p = torch.zeros_like(logits).scatter_add(1, index, torch.where(chosen, weights, 0.0))
    else:
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True) * chosen.any(1, keepdim=True)
    at = torch.where(chosen, dweights * weights, 0.0)
    return torch.zeros_like(logits).scatter_add(1, index, at) - p * inner


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h = s["x"].float() + s["residual"].float()
        rstd = torch.rsqrt(h.square().mean(1) + EPS)
        y = h * rstd[:, None] * s["weight"].float()
        out = {"h": h.to(BF16), "rstd": rstd}
        if case["quantize"]:
            out["y"], out["scale"] = _rows_to_e4m3(y)
        else:
            out["y"] = y.to(BF16)
        return out
    if op == "norm gradient":
        h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
        g = dy * s["weight"].float()
        dx = rstd * g - h * rstd * rstd * rstd * (g * h).mean(1, keepdim=True) + s["dh"].float()
        return {"dx": dx.to(BF16), "dweight": (dy * h * rstd).sum(0)}
    if op == "route":
        live = s["live"]
        if live is None:
            live = torch.ones(case["tokens"], dtype=torch.bool, device="cuda")
        weights, experts, (slots, tokens, offsets) = _routing(s["logits"], case["topk"], live)
        if case["renormalize"]:
            total = weights.sum(1, keepdim=True)
            weights = torch.where(total > 0, weights / total, 0.0)
        return {"weights": weights, "experts": experts.int(), "slots": slots.int(),
                "tokens": tokens.int(), "offsets": offsets.int()}
    if op.startswith("combine"):
        slots = s["slots"].long()
        used = slots >= 0
        rows = s["rows"].float()[slots.clamp(min=0)] * used[:, :, None]
        if op == "combine":
            return {"y": (rows * s["weights"][:, :, None]).sum(1).to(BF16)}
        dy = s["dy"].float()[:, None, :]
        dweights = (rows * dy).sum(2)
        drows = torch.zeros((slots.numel() + 1, case["dim"]), device=dy.device)
        drows[torch.where(used, slots, -1)] = dy * s["weights"][:, :, None]
        return {"drows": drows[:-1].to(BF16), "dweights": dweights,
                "dlogits": _route_gradient(dweights, s["weights"], s["experts"], s["logits"],
                                           False)}
    groups = _groups(s)
    if op == "experts gradient":
        dy, h, pre = s["dy"].float(), s["h"].float(), s["pre"].float()
        live = groups[2][:, None]
        dpre = _gated_gradient(_product(dy, s["down"].transpose(1, 2), s, groups), pre)
        dpre = torch.where(live, dpre, 0.0)
        dx = _product(dpre, s["gate_up"].transpose(1, 2), s, groups)
        ddown = _product_dw(dy, h, s, groups)
        dgate_up = _product_dw(dpre, _gathered(s["x"], s["tokens"]), s, groups)
        return {"dpre": dpre.to(BF16), "dx": dx.to(BF16), "ddown": ddown.to(BF16),
                "dgate_up": dgate_up.to(BF16)}
    if op == "experts 8-bit":
        # e4m3 stands for value * scale; the two products and the rounding of the rows
        # between them are calls of their own, each with its own rounded output
        x = s["x"].float() * s["x_scale"][:, None]
        w = s["gate_up"], s["gate_up_scale"]
        h = _gated(_product8(_gathered(x, s["tokens"]), *w, s, groups)).to(BF16)
        h8, scale = _rows_to_e4m3(h)
        y = _product8(h8.float() * scale[:, None], s["down"], s["down_scale"], s, groups)
        return {"h": h, "y": y.to(BF16)}
    pre = _product(_gathered(s["x"], s["tokens"]), s["gate_up"], s, groups)
    h = _gated(pre)
    y = _product(h, s["down"], s, groups)
    if case["train"]:
        return {"pre": pre.to(BF16), "h": h.to(BF16), "y": y.to(BF16)}
    return {"y": y.to(BF16)}


def _product8(rows, w, scale, s, groups):
    """_product with e4m3 weights: the output features' scales go on at the end."""
    return _product(rows, w, s, groups) * scale[groups[0]]


# ------------------------------------------------------------------ one pass

def run(state):
    if not own:
        return _plain(state)
    from lossless_exponent_reuse_gb300 import experts
    s, case = state, state["case"]
    op = case["op"]
    if op == "norm":
        r = experts.rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS,
                            quantize=case["quantize"])
        out = {"y": r.y, "h": r.h, "rstd": r.rstd}
        if case["quantize"]:
            out["scale"] = r.scale
        return out
    if op == "norm gradient":
        dx, dweight = experts.rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["weight"],
                                               dh=s["dh"])
        return {"dx": dx, "dweight": dweight}
    if op == "route":
        r = experts.route(s["logits"], case["topk"], renormalize=case["renormalize"],
                          token_mask=s["live"])
        return {"weights": r.weights, "experts": r.experts, "slots": r.slots,
                "tokens": r.tokens, "offsets": r.offsets}
    if op == "combine":
        return {"y": experts.combine(s["rows"], s["slots"], s["weights"])}
    if op == "combine gradient":
        drows, dweights = experts.combine_backward(s["dy"], s["rows"], s["slots"], s["weights"],
                                                   s["offsets"])
        dlogits = experts.route_backward(dweights, s["weights"], s["experts"], s["logits"])
        return {"drows": drows, "dweights": dweights, "dlogits": dlogits}
    off = s["offsets"]
    if op == "experts gradient":
        dpre = experts.mm_dx(s["dy"], s["down"], off, gated=s["pre"])
        dx = experts.mm_dx(dpre, s["gate_up"], off)
        ddown = experts.mm_dw(s["dy"], s["h"], off)
        dgate_up = experts.mm_dw(dpre, s["x"], off, tokens=s["tokens"])
        return {"dpre": dpre, "dx": dx, "ddown": ddown, "dgate_up": dgate_up}
    if op == "experts 8-bit":
        h = experts.mm_gated(s["x"], s["gate_up"], off, tokens=s["tokens"],
                             x_scale=s["x_scale"], w_scale=s["gate_up_scale"])
        h8, h_scale = experts.quantize_rows(h)
        y = experts.mm(h8, s["down"], off, x_scale=h_scale, w_scale=s["down_scale"])
        return {"h": h, "y": y}
    if case["train"]:
        h, pre = experts.mm_gated(s["x"], s["gate_up"], off, tokens=s["tokens"], keep=True)
        return {"pre": pre, "h": h, "y": experts.mm(h, s["down"], off)}
    h = experts.mm_gated(s["x"], s["gate_up"], off, tokens=s["tokens"])
    return {"y": experts.mm(h, s["down"], off)}


def work(case):
    op, T = case["op"], case["tokens"]
    if op == "norm":
        n = T * case["dim"]
        return {"bytes": n * (7 if case["quantize"] else 8) + 2 * case["dim"] + 4 * T,
                "flops": 6 * n}
    if op == "norm gradient":
        n = T * case["dim"]
        return {"bytes": 8 * n + 6 * case["dim"] + 4 * T, "flops": 10 * n}
    E, k = case["experts"], case["topk"]
    R = T * k
    if op == "route":
        size = 4 if case["logits"] == "f32" else 2
        return {"bytes": T * E * size + 16 * R + 4 * (E + 1), "flops": 4 * T * E}
    if op == "combine":
        return {"bytes": 2 * R * case["dim"] + 2 * T * case["dim"] + 8 * R,
                "flops": 2 * R * case["dim"]}
    if op == "combine gradient":
        return {"bytes": 4 * R * case["dim"] + 2 * T * case["dim"] + 16 * R + 8 * T * E,
                "flops": 3 * R * case["dim"]}
    D, F = case["dim"], case["ff"]
    R = round(R * (1 - case["masked"]))
    # experts that at least one token chose, were the choice uniform
    touched = min(R, E * (1 - (1 - min(1.0, k / E)) ** T))
    if op == "experts gradient":
        return {"bytes": 2 * (touched + E) * 3 * F * D
                + 2 * (2 * R * D + T * D + 5 * R * F), "flops": 12 * R * F * D}
    if op == "experts 8-bit":
        return {"bytes": touched * 3 * F * D + T * D + 2 * R * F + 2 * R * D,
                "flops": 6 * R * F * D}
    kept = 6 * R * F if case["train"] else 0
    return {"bytes": 2 * touched * 3 * F * D + 2 * T * D + kept + 2 * R * D,
            "flops": 6 * R * F * D}


# ------------------------------------------------------- definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, T = case["op"], case["tokens"]
    d = {n: v.double() for n, v in s.items()
         if torch.is_tensor(v) and v.is_floating_point() and v.dim() != 3}
    if op == "norm":
        h = d["x"] + d["residual"]
        rstd = 1 / ((h * h).sum(1) / case["dim"] + EPS).sqrt()
        y = torch.einsum("td,t,d->td", h, rstd, d["weight"])
        out = {"h": h, "rstd": rstd}
        if case["quantize"]:
            scale = y.abs().max(1).values.clamp(min=TINY) / E4M3_MAX
            out.update(scale=scale, y=torch.einsum("td,t->td", y, 1 / scale))
        else:
            out["y"] = y
        return out
    if op == "norm gradient":
        # y_i = w_i h_i r with r = (mean(h^2) + eps)^(-1/2): dr/dh_i = -r^3 h_i / D
        h, dy, r = d["h"], d["dy"], d["rstd"]
        dr = torch.einsum("td,td,d->t", dy, h, d["weight"])
        dx = (torch.einsum("td,d,t->td", dy, d["weight"], r)
              - torch.einsum("td,t->td", h, dr * r ** 3 / case["dim"]) + d["dh"])
        return {"dx": dx, "dweight": torch.einsum("td,td,t->d", dy, h, r)}
    k = case["topk"]
    if op == "route":
        l = d["logits"]
        p = torch.softmax(l, 1)
        # the k largest, ties to the lowest index: count what stands before each logit
        E = case["experts"]
        index = torch.arange(E, device=l.device)
        lower = index[None, :] < index[:, None]
        weights = torch.zeros(T, k, dtype=torch.float64, device=l.device)
        for t in range(0, T, 1024):
            b = l[t:t + 1024]
            rank = ((b[:, None, :] > b[:, :, None])
                    | ((b[:, None, :] == b[:, :, None]) & lower)).sum(2)
            at = torch.argsort(rank, 1)[:, :k]
            weights[t:t + 1024] = p[t:t + 1024].gather(1, at)
        if case["renormalize"]:
            weights /= weights.sum(1, keepdim=True)
        if s["live"] is not None:
            weights[~s["live"]] = 0
        return {"weights": weights, "experts": None, "slots": None, "tokens": None,
                "offsets": None}
    if op.startswith("combine"):
        slots, w = s["slots"].long(), d["weights"]
        rows = torch.cat([d["rows"], torch.zeros_like(d["rows"][:1])])
        if op == "combine":
            y = torch.zeros(T, case["dim"], dtype=torch.float64, device=rows.device)
            for j in range(k):
                y += w[:, j:j + 1] * rows[slots[:, j]]     # -1: the row of zeros
            return {"y": y}
        dw, drows = torch.zeros_like(w), torch.zeros_like(rows)
        for j in range(k):
            dw[:, j] = (d["dy"] * rows[slots[:, j]]).sum(1)
            drows[slots[:, j]] = w[:, j:j + 1] * d["dy"]
        # w_j = p_(e_j): dw_j / dl_i = p_(e_j) ([i = e_j] - p_i)
        p = torch.softmax(d["logits"], 1)
        dl = torch.zeros_like(p)
        for j in range(k):
            e = s["experts"][:, j].long()
            on = (e >= 0).double()[:, None]
            hot = torch.nn.functional.one_hot(e.clamp(min=0), case["experts"]).double()
            dl += on * (dw[:, j:j + 1] * p.gather(1, e.clamp(min=0)[:, None])) * (hot - p)
        return {"drows": drows[:-1], "dweights": dw, "dlogits": dl}

    D, F, R = case["dim"], case["ff"], T * k
    bounds = s["offsets"].tolist()
    new = {n: torch.zeros(R, m, dtype=torch.float64, device="cuda")
           for n, m in (("pre", 2 * F), ("h", F), ("y", D), ("dpre", 2 * F), ("dx", D))}
    grads = {}
    if op == "experts gradient":
        grads = {"ddown": torch.zeros(case["experts"], D, F, dtype=torch.float64, device="cuda"),
                 "dgate_up": torch.zeros(case["experts"], 2 * F, D, dtype=torch.float64,
                                         device="cuda")}
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if a == b:
            continue
        gu, dn = s["gate_up"][e].double(), s["down"][e].double()
        at = s["tokens"][a:b].long()
        x = d["x"][at]
        if op == "experts 8-bit":
            x = x * d["x_scale"][at][:, None]
            gu = gu * s["gate_up_scale"][e].double()[:, None]
            dn = dn * s["down_scale"][e].double()[:, None]
            pre = x @ gu.T
            h = pre[:, :F] / (1 + torch.exp(-pre[:, :F])) * pre[:, F:]
            new["h"][a:b] = h
            h = h.to(BF16).double()            # the first product's output type
            scale = h.abs().max(1, keepdim=True).values.clamp(min=TINY) / E4M3_MAX
            new["y"][a:b] = ((h / scale).to(E4M3).double() * scale) @ dn.T
        elif op == "experts":
            pre = x @ gu.T
            h = pre[:, :F] / (1 + torch.exp(-pre[:, :F])) * pre[:, F:]
            new["pre"][a:b], new["h"][a:b], new["y"][a:b] = pre, h, h @ dn.T
        else:
            dy, pre = d["dy"][a:b], d["pre"][a:b]
            dh = dy @ dn
            gate, up = pre[:, :F], pre[:, F:]
            sig = 1 / (1 + torch.exp(-gate))
            dpre = torch.cat([dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig], 1)
            new["dpre"][a:b], new["dx"][a:b] = dpre, dpre @ gu
            grads["ddown"][e], grads["dgate_up"][e] = dy.T @ d["h"][a:b], dpre.T @ x
    if op == "experts gradient":
        return {"dpre": new["dpre"], "dx": new["dx"], **grads}
    if op == "experts 8-bit":
        return {"h": new["h"], "y": new["y"]}
    return {n: new[n] for n in (("pre", "h", "y") if case["train"] else ("y",))}
