"""Norm, route and combine of the mixture-of-experts layer against their
formulas in 64 bits, at the sizes, strides and masks where they can go wrong."""
import math

import pytest
import torch

import moe_reference as ref
from lossless_exponent_reuse_gb300 import ciera, experts

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def rand(*shape, seed=0, scale=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000 * len(shape) + sum(shape))
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def strided(t, kind):
    """The same matrix in other memory: a column slice of a wider one, at an
    even or an odd column."""
    if kind == "plain":
        return t
    pad = {"wide": 8, "odd": 3}[kind]
    wide = torch.full((t.shape[0], t.shape[1] + 2 * pad), float("nan"), dtype=t.dtype,
                      device=t.device)
    wide[:, pad:pad + t.shape[1]] = t
    return wide[:, pad:pad + t.shape[1]]


SIZES = [(0, 8), (1, 1), (1, 2048), (3, 7), (5, 1000), (2, 1001), (33, 1536), (700, 264),
         (1300, 40), (4, 8200), (2, 40000)]


# ---- norm ----------------------------------------------------------------

@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("with_residual", [True, False])
def test_norm(rows, dim, with_residual, kind):
    x, w = rand(rows, dim), rand(dim, seed=1) + 1
    res = rand(rows, dim, seed=2, scale=3.0) if with_residual else None
    s, rstd, y = ref.norm(x, w, res, 1e-6)
    # the sum of squares has `dim` positive terms; rstd halves its relative error
    e_rstd = (dim + 8) * ref.U_F32
    sized = s if res is None else x.double().abs() + res.double().abs()
    e_y = y.abs() * (e_rstd + 4 * ref.U_F32) + (sized * rstd[:, None] * w.double().abs()
                                                * ref.U_F32)
    xs = strided(x, kind)
    rs = None if res is None else strided(res, kind)
    r = experts.rmsnorm(xs, w, residual=rs, eps=1e-6)
    ref.within(r.rstd, rstd, 0.0, "rstd", rounded=e_rstd)
    ref.within(r.y, y, e_y, "y")
    ref.within(r.h, s, sized * ref.U_F32, "h")
    if res is None:
        assert r.h is xs
    q = experts.rmsnorm(xs, w, residual=rs, eps=1e-6, quantize=True)
    assert q.y.dtype == torch.float8_e4m3fn
    if dim:
        scale, code = ref.quantize(y)
        e_row = (e_y / scale[:, None])
        # the scale's error is that of the row's largest value
        ref.within(q.scale, scale, e_y.amax(1) / ref.E4M3_MAX, "scale", rounded=4 * ref.U_F32)
        slack = e_row + code.abs() * (e_y.amax(1) / ref.E4M3_MAX / scale)[:, None] \
            + code.abs() * 8 * ref.U_F32 + 2.0 ** -10
        ref.within(q.y.float(), code, slack, "e4m3", rounded=2.0 ** -4)
    torch.testing.assert_close(q.h, r.h, rtol=0, atol=0)


def guarded(t, at):
    """The values at element ``at`` of a flat buffer, others around them; (view, buffer)."""
    flat = torch.full((t.numel() + at + 24,), 7.0, device="cuda").to(t.dtype)
    flat[at:at + t.numel()] = t.reshape(-1)
    return flat[at:at + t.numel()].view(t.shape), flat


def untouched(flat, at, n):
    return (flat[:at].float() == 7).all() and (flat[at + n:].float() == 7).all()


@pytest.mark.parametrize("at", range(8))
@pytest.mark.parametrize("dim", [769, 1001, 2047, 4099, 9001])
def test_norm_of_odd_rows_that_start_anywhere(dim, at):
    """All matrices at the same place behind a 16-byte boundary; nothing is
    written outside the rows."""
    rows = 5
    x, w = rand(rows, dim), rand(dim, seed=1) + 1
    res = rand(rows, dim, seed=2, scale=3.0)
    s, rstd, y = ref.norm(x, w, res, 1e-6)
    e_rstd = (dim + 8) * ref.U_F32
    sized = x.double().abs() + res.double().abs()
    e_y = y.abs() * (e_rstd + 4 * ref.U_F32) + (sized * rstd[:, None] * w.double().abs()
                                                * ref.U_F32)
    (xs, _), (rs, _) = guarded(x, at), guarded(res, at)
    for kind, dtype in ((experts.BF16, BF16), (experts.E4M3, torch.float8_e4m3fn)):
        ys, y_flat = guarded(torch.zeros(rows, dim, dtype=BF16, device="cuda").to(dtype), at)
        hs, h_flat = guarded(torch.zeros_like(x), at)
        scale, r = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
        st = ciera.lib().ciera_rmsnorm(
            xs.data_ptr(), dim, rs.data_ptr(), dim, w.data_ptr(), rows, dim, 1e-6, ys.data_ptr(),
            kind, scale.data_ptr() if kind == experts.E4M3 else None, hs.data_ptr(), r.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
        assert st == ciera.OK
        assert untouched(y_flat, at, rows * dim) and untouched(h_flat, at, rows * dim)
        ref.within(r, rstd, 0.0, "rstd", rounded=e_rstd)
        ref.within(hs, s, sized * ref.U_F32, "h")
        if kind == experts.BF16:
            ref.within(ys, y, e_y, "y")
        else:
            want, code = ref.quantize(y)
            ref.within(scale, want, e_y.amax(1) / ref.E4M3_MAX, "scale", rounded=4 * ref.U_F32)
            slack = e_y / want[:, None] + code.abs() * (e_y.amax(1) / ref.E4M3_MAX / want)[:, None] \
                + code.abs() * 8 * ref.U_F32 + 2.0 ** -10
            ref.within(ys.float(), code, slack, "e4m3", rounded=2.0 ** -4)
    # rows to e4m3 as they are
    ys, y_flat = guarded(torch.zeros(rows, dim, device="cuda").to(torch.float8_e4m3fn), at)
    st = ciera.lib().ciera_quantize_rows(xs.data_ptr(), dim, rows, dim, ys.data_ptr(),
                                         scale.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == ciera.OK and untouched(y_flat, at, rows * dim)
    want, code = ref.quantize(x.double())
    ref.within(scale, want, 0.0, "scale", rounded=2 * ref.U_F32)
    ref.within(ys.float(), code, code.abs() * 8 * ref.U_F32 + 2.0 ** -10, "e4m3",
               rounded=2.0 ** -4)


def test_norm_of_odd_zero_rows():
    """Nothing behind a row's end counts, even where zeros give no number."""
    x = torch.zeros(9, 1001, dtype=BF16, device="cuda")
    w = torch.ones(1001, dtype=BF16, device="cuda")
    r = experts.rmsnorm(x, w, eps=1e-6, quantize=True)
    assert (r.y.float() == 0).all() and torch.isfinite(r.scale).all()
    x[:, 1000] = 1.0
    r = experts.rmsnorm(x, w, eps=0.0, quantize=True)
    assert (r.y[:, 1000].float() == 448).all() and (r.y[:, :1000].float() == 0).all()


def test_norm_of_zeros_infinities_and_nan():
    w = torch.ones(64, dtype=BF16, device="cuda")
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] = 1e-38                                    # squares underflow
    r = experts.rmsnorm(x, w, eps=0.0)
    assert torch.isnan(r.y[0]).all()                # 0 times an infinite rstd
    assert r.y[1, 0] == 0 and torch.isnan(r.y[1, 3])
    assert torch.isnan(r.y[2]).all()
    r = experts.rmsnorm(x, w, eps=1e-6, quantize=True)
    assert (r.y[0].float() == 0).all() and torch.isfinite(r.scale[0]) and r.scale[0] > 0
    assert torch.isnan(r.scale[1]) and torch.isnan(r.scale[2])
    assert torch.isfinite(r.y[3].float() * r.scale[3]).all()
    y, scale = experts.quantize_rows(x)
    assert (y[0].float() == 0).all()
    assert torch.isnan(scale[1]) and torch.isnan(scale[2]) and torch.isfinite(scale[3])


def test_norm_keeps_the_sum_in_place_of_the_residual():
    import ctypes
    x, res, w = rand(5, 48), rand(5, 48, seed=3), rand(48, seed=4)
    want = experts.rmsnorm(x, w, residual=res)
    y, rstd = torch.empty_like(x), torch.empty(5, device="cuda")
    h = res.clone()
    st = ciera.lib().ciera_rmsnorm(x.data_ptr(), 48, h.data_ptr(), 48, w.data_ptr(), 5, 48, 1e-6,
                                   y.data_ptr(), experts.BF16, None, h.data_ptr(),
                                   rstd.data_ptr(), ctypes.c_void_p(
                                       torch.cuda.current_stream().cuda_stream))
    assert st == ciera.OK
    assert torch.equal(h, want.h) and torch.equal(y, want.y) and torch.equal(rstd, want.rstd)


@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("rows,dim", SIZES)
def test_quantize_rows(rows, dim, kind):
    x = rand(rows, dim, scale=5.0)
    y, scale = experts.quantize_rows(strided(x, kind))
    want, code = ref.quantize(x.double())
    ref.within(scale, want, 0.0, "scale", rounded=2 * ref.U_F32)
    ref.within(y.float(), code, code.abs() * 6 * ref.U_F32 + 2.0 ** -10, "e4m3",
               rounded=2.0 ** -4)


@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("with_dh", [True, False])
def test_norm_gradient(rows, dim, with_dh, kind):
    h, w = rand(rows, dim, seed=5, scale=2.0), rand(dim, seed=6) + 1
    dy = rand(rows, dim, seed=7)
    dh = rand(rows, dim, seed=8) if with_dh else None
    # the formula's gradient, by differentiating the definition in 64 bits
    hd, wd = h.double().requires_grad_(), w.double().requires_grad_()
    r = (hd * hd).mean(1).add(1e-6) ** -0.5 if rows and dim else torch.ones(rows).cuda().double()
    (hd * r[:, None] * wd * dy.double()).sum().backward()
    rstd = r.detach().float()
    dx, dw = experts.rmsnorm_backward(strided(dy, kind), strided(h, kind), rstd, w,
                                      dh=None if dh is None else strided(dh, kind))
    if not rows:
        assert dx.shape == (rows, dim) and (dw == 0).all()
        return
    rd = r.detach()[:, None]
    g = dy.double().abs() * w.double().abs()
    size = rd * g + h.double().abs() * rd ** 3 * (g * h.double().abs()).mean(1, keepdim=True)
    want = hd.grad
    if dh is not None:
        want = want + dh.double()
        size = size + dh.double().abs()
    ref.within(dx, want, size * (dim + 16) * ref.U_F32, "dx")
    terms = (dy.double().abs() * h.double().abs() * rd).sum(0)
    ref.within(dw, wd.grad, terms * (rows + 8) * ref.U_F32, "dweight", rounded=ref.U_F32)
    # the same call again gives the same bits
    again = experts.rmsnorm_backward(strided(dy, kind), strided(h, kind), rstd, w,
                                     dh=None if dh is None else strided(dh, kind))
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("at", range(8))
@pytest.mark.parametrize("rows,dim", [(3, 129), (5000, 129), (3000, 511), (2500, 1001),
                                      (1500, 2047), (700, 5001), (400, 9001)])
def test_norm_gradient_of_odd_rows_that_start_anywhere(rows, dim, at):
    """All matrices at the same place behind a 16-byte boundary, more rows than
    blocks at once; nothing is written outside the rows."""
    h, w = rand(rows, dim, seed=5, scale=2.0), rand(dim, seed=6) + 1
    dy, dh = rand(rows, dim, seed=7), rand(rows, dim, seed=8)
    hd, wd, dyd = h.double(), w.double(), dy.double()
    rd = ((hd * hd).mean(1, keepdim=True) + 1e-6) ** -0.5
    rstd = rd[:, 0].float()
    g = dyd * wd
    want = rd * g - hd * rd ** 3 * (g * hd).mean(1, keepdim=True) + dh.double()
    size = rd * g.abs() + hd.abs() * rd ** 3 * (g * hd).abs().mean(1, keepdim=True) \
        + dh.double().abs()
    (dys, _), (hs, _), (dhs, _) = (guarded(t, at) for t in (dy, h, dh))
    dxs, dx_flat = guarded(torch.zeros_like(dy), at)
    dw = torch.zeros(dim, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    ws = experts.workspace(0, s, tokens=rows, dim=dim)
    st = ciera.lib().ciera_rmsnorm_backward(
        dys.data_ptr(), dim, hs.data_ptr(), dim, rstd.data_ptr(), w.data_ptr(), dhs.data_ptr(),
        dim, rows, dim, dxs.data_ptr(), dw.data_ptr(), ws.data_ptr(), ws.numel(), s)
    assert st == ciera.OK and untouched(dx_flat, at, rows * dim)
    ref.within(dxs, want, size * (dim + 16) * ref.U_F32, "dx")
    terms = (dyd.abs() * hd.abs() * rd).sum(0)
    ref.within(dw, (dyd * hd * rd).sum(0), terms * (rows + 8) * ref.U_F32, "dweight",
               rounded=ref.U_F32)


def test_norm_gradient_against_differences():
    rows, dim = 6, 96
    x, w, dy = rand(rows, dim, seed=9), rand(dim, seed=10) + 1, rand(rows, dim, seed=11)
    kept = experts.rmsnorm(x, w)
    dx, dw = experts.rmsnorm_backward(dy, kept.h, kept.rstd, w)
    along = rand(rows, dim, seed=12).double()
    loss = lambda v: (ref.norm(v, w, None, 1e-6)[2] * dy.double()).sum()
    step = 1e-4
    slope = (loss(x.double() + step * along) - loss(x.double() - step * along)) / (2 * step)
    got = (dx.double() * along).sum()
    # each dx is off by 2^-8 relative at most, and the quotient by O(step^2)
    assert abs(got - slope) <= (dx.double().abs() * along.abs()).sum() * 2.0 ** -8 + 1e-5
    loss_w = lambda v: (ref.norm(x, v, None, 1e-6)[2] * dy.double()).sum()
    wa = rand(dim, seed=13).double()
    slope = (loss_w(w.double() + step * wa) - loss_w(w.double() - step * wa)) / (2 * step)
    assert abs((dw.double() * wa).sum() - slope) <= (dw.double().abs() * wa.abs()).sum() * 1e-5 \
        + 1e-7


# ---- route ---------------------------------------------------------------

ROUTES = [(1, 1, 1), (1, 64, 8), (7, 8, 8), (63, 60, 4), (64, 100, 6), (65, 128, 8), (500, 33, 2),
          (200, 256, 32), (130, 1024, 3), (1, 1000, 32), (5000, 16, 1)]


def check_routing(r, logits, k, renormalize, mask=None):
    chosen, weights, slots, tokens, offsets = ref.route(logits, k, mask)
    assert r.experts.tolist() == chosen
    assert r.slots.tolist() == slots
    assert r.tokens.tolist() == tokens
    assert r.offsets.tolist() == offsets
    want = torch.tensor(weights, dtype=torch.float64, device="cuda").reshape(r.weights.shape)
    if renormalize:
        total = want.sum(1, keepdim=True)
        want = torch.where(total > 0, want / total, 0.0)
    # exp within 2 ulp of an argument rounded at |l - max| <= 32, sums of E terms
    E = logits.shape[1]
    ref.within(r.weights, want, 0.0, "weights", rounded=(E + 96) * ref.U_F32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route(T, E, k, renormalize, dtype):
    logits = rand(T, E, seed=14, dtype=dtype)
    r = experts.route(logits, k, renormalize=renormalize)
    check_routing(r, logits, k, renormalize)
    wide = strided(logits, "odd") if E > 1 else logits
    for a, b in zip(r, experts.route(wide, k, renormalize=renormalize)):
        assert torch.equal(a, b)


def test_route_ties_masks_and_minus_infinity():
    T, E, k = 150, 24, 4
    logits = (rand(T, E, seed=15, dtype=F32) * 2).round()      # many ties
    logits[3] = 0.0
    logits[4, ::2] = -0.0                                      # -0 and 0 tie
    logits[4, 1::2] = 0.0
    logits[5] = -math.inf                                      # nothing to choose
    logits[6] = -math.inf
    logits[6, 7] = -3.0                                        # one to choose
    logits[7, :22] = -math.inf
    logits[8] = torch.finfo(F32).min                           # lowest finite value: chosen
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[10:20] = False
    for renormalize in (False, True):
        r = experts.route(logits, k, renormalize=renormalize, token_mask=mask)
        check_routing(r, logits, k, renormalize, mask)
        assert (r.experts[5] == -1).all() and (r.weights[5] == 0).all()
        assert r.experts[6].tolist() == [7, -1, -1, -1] and r.weights[6, 0] == 1
        assert r.experts[8].tolist() == [0, 1, 2, 3]
        dl = experts.route_backward(torch.ones_like(r.weights), r.weights, r.experts, logits,
                                    renormalize=renormalize)
        assert torch.isfinite(dl).all()
        assert (dl[5] == 0).all() and (dl[10:20] == 0).all()
    everyone = torch.zeros(T, dtype=torch.uint8, device="cuda")
    r = experts.route(logits, k, token_mask=everyone)
    assert (r.offsets == 0).all() and (r.tokens == -1).all() and (r.slots == -1).all()


def test_route_nan_goes_first_and_poisons_its_token_only():
    logits = rand(4, 40, seed=16, dtype=F32)
    logits[2, 30] = float("nan")
    r = experts.route(logits, 3)
    assert int(r.experts[2, 0]) == 30
    assert torch.isnan(r.weights[2]).all()
    assert torch.isfinite(r.weights[[0, 1, 3]]).all()
    assert int(r.offsets[-1]) == 12


def test_route_all_tokens_to_one_expert_and_no_tokens():
    logits = torch.zeros(1000, 8, device="cuda")
    logits[:, 5] = 9.0
    r = experts.route(logits, 1)
    assert r.offsets.tolist() == [0] * 6 + [1000] * 3
    assert torch.equal(r.tokens, torch.arange(1000, dtype=torch.int32, device="cuda"))
    r = experts.route(torch.empty(0, 8, device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 9 and r.tokens.numel() == 0


def test_route_many_tokens():
    T, E, k = 40000, 64, 8
    logits = rand(T, E, seed=17, dtype=F32)
    r = experts.route(logits, k)
    order = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(r.experts, order.int())
    by, at = torch.sort(order.reshape(-1), stable=True)
    assert torch.equal(r.tokens, (at // k).int())
    slots = torch.empty(T * k, dtype=torch.int32, device="cuda")
    slots[at] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    assert torch.equal(r.slots.reshape(-1), slots)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route_gradient(T, E, k, renormalize, dtype):
    logits = rand(T, E, seed=18, dtype=dtype)
    r = experts.route(logits, k, renormalize=renormalize)
    dw = rand(T, k, seed=19, dtype=F32)
    l = logits.double().requires_grad_()
    w = torch.softmax(l, 1).gather(1, r.experts.long())
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    (w * dw.double()).sum().backward()
    dl = experts.route_backward(dw, r.weights, r.experts, logits, renormalize=renormalize)
    assert dl.dtype == dtype
    size = (w.detach() * dw.double().abs()).sum(1, keepdim=True).expand(T, E)
    ref.within(dl, l.grad, size * (2 * E + 200) * ref.U_F32, "dlogits",
               rounded=ref.U_BF16 if dtype == BF16 else ref.U_F32)


def test_route_gradient_against_differences():
    T, E, k = 5, 24, 4
    logits, dw = rand(T, E, seed=20, dtype=F32), rand(T, k, seed=21, dtype=F32)
    along = rand(T, E, seed=22, dtype=F32).double()
    for renormalize in (False, True):
        r = experts.route(logits, k, renormalize=renormalize)

        def loss(l):
            w = torch.softmax(l, 1).gather(1, r.experts.long())
            if renormalize:
                w = w / w.sum(1, keepdim=True)
            return (w * dw.double()).sum()

        step = 1e-5
        l = logits.double()
        slope = (loss(l + step * along) - loss(l - step * along)) / (2 * step)
        dl = experts.route_backward(dw, r.weights, r.experts, logits, renormalize=renormalize)
        assert abs((dl.double() * along).sum() - slope) <= 1e-5


# ---- combine ---------------------------------------------------------------

COMBINES = [(1, 8, 2048, 64), (3, 2, 7, 5), (333, 8, 1000, 64), (40, 1, 1001, 8),
            (17, 32, 136, 40), (2, 3, 9000, 4), (700, 4, 64, 16)]


@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("T,k,dim,E", COMBINES)
def test_combine_and_its_gradient(T, k, dim, E, kind):
    mask = torch.rand(T, generator=torch.Generator().manual_seed(T)) > 0.2
    r = experts.route(rand(T, E, seed=23, dtype=F32), k, token_mask=mask.cuda())
    rows = rand(T * k, dim, seed=24)
    rows[int(r.offsets[-1]):] = float("nan")            # unused rows are not read
    dy = rand(T, dim, seed=25)
    s = r.slots.long()
    used = s >= 0
    picked = torch.where(used[:, :, None], rows.double()[s.clamp(min=0)], 0.0)
    w = r.weights.double()[:, :, None]
    u = (k + 2) * ref.U_F32
    y = experts.combine(strided(rows, kind), r.slots, r.weights)
    ref.within(y, (picked * w).sum(1), (picked * w).abs().sum(1) * u, "y")
    y = experts.combine(strided(rows, kind), r.slots)
    ref.within(y, picked.sum(1), picked.abs().sum(1) * u, "sum")
    drows, dweights = experts.combine_backward(strided(dy, kind), strided(rows, kind), r.slots,
                                               r.weights, r.offsets)
    want = torch.zeros(T * k, dim, dtype=torch.float64, device="cuda")
    want[s[used]] = (w * dy.double()[:, None, :])[used]
    ref.within(drows, want, want.abs() * 2 * ref.U_F32, "drows")
    terms = picked * dy.double()[:, None, :]
    ref.within(dweights, terms.sum(2), terms.abs().sum(2) * (dim + 2) * ref.U_F32, "dweights",
               rounded=ref.U_F32)


@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("T,R,dim", [(1, 8, 2048), (40, 0, 16), (40, 333, 1001), (7, 100, 136),
                                     (5, 9, 1)])
def test_gather_rows(T, R, dim, kind):
    x = rand(T, dim, seed=29)
    tokens = torch.randint(-1, T + 1, (R,), generator=torch.Generator().manual_seed(R),
                           dtype=torch.int32).cuda()
    some = (tokens >= 0) & (tokens < T)
    at = tokens.long().clamp(0, T - 1)
    want = torch.where(some[:, None], x[at], 0.0)
    assert torch.equal(experts.gather_rows(strided(x, kind), tokens), want)
    x8, scale = experts.quantize_rows(x)
    y8, y_scale = experts.gather_rows(x8, tokens, x_scale=scale)
    assert torch.equal(y8.view(torch.uint8), torch.where(some[:, None], x8.view(torch.uint8)[at],
                                                         0).to(torch.uint8))
    assert torch.equal(y_scale, torch.where(some, scale[at], 0.0))


def test_combine_takes_indexes_outside_for_none():
    rows = rand(6, 16, seed=26)
    slots = torch.tensor([[0, 6], [-5, 2 ** 30], [5, -1]], dtype=torch.int32, device="cuda")
    w = torch.ones(3, 2, device="cuda")
    y = experts.combine(rows, slots, w)
    assert torch.equal(y[0], rows[0]) and (y[1] == 0).all() and torch.equal(y[2], rows[5])
    offsets = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    drows, dweights = experts.combine_backward(rows[:3], rows, slots, w, offsets)
    assert (dweights[0, 1] == 0) and (dweights[1] == 0).all()
    assert torch.equal(drows[0], rows[0]) and torch.equal(drows[5], rows[2])


def test_rows_on_another_stream():
    """Calls on a side stream, and outputs freed there, see their own inputs."""
    side = torch.cuda.Stream()
    x, w = rand(4096, 2048, seed=27), rand(2048, seed=28)
    want = experts.rmsnorm(x, w).y
    torch.cuda.synchronize()
    for _ in range(5):
        got = experts.rmsnorm(x, w, stream=side).y
        experts.rmsnorm(x, w, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want)


def test_a_graph_outlives_its_workspace():
    """A captured call keeps its scratch memory when a larger call wants more."""
    h, dy, w = rand(64, 256, seed=30), rand(64, 256, seed=31), rand(256, seed=32)
    rstd = torch.ones(64, device="cuda")
    want = experts.rmsnorm_backward(dy, h, rstd, w)
    side = torch.cuda.Stream()
    experts.rmsnorm_backward(dy, h, rstd, w, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dx, dw = experts.rmsnorm_backward(dy, h, rstd, w)
    big = rand(3000, 2048, seed=33)
    experts.rmsnorm_backward(big, big, torch.ones(3000, device="cuda"), rand(2048, seed=34),
                             stream=side)
    side.synchronize()
    filler = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(8)]
    dw.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    assert all((f == 3.0).all() for f in filler)


@pytest.mark.parametrize("dim", [16, 17])
@pytest.mark.parametrize("ends,used", [([4, 2], 4), ([], 0), ([99, 3], 8), ([-3, -1], 0),
                                       ([6, 6], 6), ([1] * 1023 + [5], 5)])
def test_combine_gradient_reads_offsets_as_the_products_do(ends, used, dim):
    """Rows from the highest offset on are zeroed, and no row that has a slot;
    offsets[0] is not read."""
    rows, dy = rand(8, dim, seed=40), rand(8, dim, seed=41)
    slots = torch.arange(8, dtype=torch.int32, device="cuda")[:, None].clone()
    slots[used:] = -1
    offsets = torch.tensor([2 ** 30, *ends], dtype=torch.int32, device="cuda")
    w = torch.full((8, 1), 0.5, device="cuda")
    drows, dweights = experts.combine_backward(dy, rows, slots, w, offsets)
    assert torch.equal(drows[:used], (dy[:used].float() * 0.5).to(BF16))
    assert (drows[used:] == 0).all() and (dweights[used:] == 0).all()


@pytest.mark.parametrize("rows", [1, 5, 3000])
def test_rows_of_no_columns(rows):
    """Their scales are those of zeros and are written; memory that held something
    else before is behind them."""
    x, w = rand(rows, 0, seed=50), rand(0, seed=51)
    tiny = torch.full((rows,), ref.TINY, device="cuda") / ref.E4M3_MAX
    for res in (None, x):
        dirty = [torch.full((rows,), 7.0, device="cuda") for _ in range(4)]
        del dirty
        q = experts.rmsnorm(x, w, residual=res, quantize=True)
        assert torch.equal(q.scale, tiny) and q.rstd.isnan().all()
        dirty = [torch.full((rows,), 7.0, device="cuda") for _ in range(4)]
        del dirty
        assert experts.rmsnorm(x, w, residual=res).rstd.isnan().all()
    dirty = [torch.full((rows,), 7.0, device="cuda") for _ in range(4)]
    del dirty
    y, scale = experts.quantize_rows(x)
    assert y.shape == (rows, 0) and torch.equal(scale, tiny)
    y, scale = experts.quantize_rows(x.view(1, rows, 0))
    assert y.shape == (1, rows, 0) and torch.equal(scale, tiny[None])
    tokens = torch.tensor([0, -1, rows - 1], dtype=torch.int32, device="cuda")
    dirty = [torch.full((3,), 7.0, device="cuda") for _ in range(4)]
    del dirty
    _, got = experts.gather_rows(y[0], tokens, x_scale=scale[0])
    assert torch.equal(got, torch.stack([tiny[0], tiny[0] * 0, tiny[0]]))


@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("rows,dim", [(500, 5120), (500, 7168), (400, 8200), (320, 16384),
                                      (900, 12290), (800, 17000)])
def test_norm_gradient_of_wide_rows_with_several_a_block(rows, dim, kind):
    h, w = rand(rows, dim, seed=52, scale=2.0), rand(dim, seed=53) + 1
    dy, dh = rand(rows, dim, seed=54), rand(rows, dim, seed=55)
    hd, dyd = h.double(), dy.double()
    rd = ((hd * hd).mean(1, keepdim=True) + 1e-6) ** -0.5
    g = dyd * w.double()
    want = rd * g - hd * rd ** 3 * (g * hd).mean(1, keepdim=True) + dh.double()
    size = rd * g.abs() + hd.abs() * rd ** 3 * (g * hd).abs().mean(1, keepdim=True) \
        + dh.double().abs()
    dx, dw = experts.rmsnorm_backward(strided(dy, kind), strided(h, kind), rd[:, 0].float(), w,
                                      dh=strided(dh, kind))
    ref.within(dx, want, size * (dim + 16) * ref.U_F32, "dx")
    terms = (dyd.abs() * hd.abs() * rd).sum(0)
    ref.within(dw, (dyd * hd * rd).sum(0), terms * (rows + 8) * ref.U_F32, "dweight",
               rounded=ref.U_F32)


def test_route_refuses_more_choices_than_it_makes():
    logits = rand(3, 64, seed=60, dtype=F32)
    for topk, most in ((0, 32), (33, 32), (64, 32), (-1, 32)):
        with pytest.raises(ValueError, match=f"1..{most}"):
            experts.route(logits, topk)
    with pytest.raises(ValueError, match="1..8"):
        experts.route(logits[:, :8], 9)
    assert experts.route(logits, 32).weights.shape == (3, 32)
