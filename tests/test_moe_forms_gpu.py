"""Forms of the grouped products that a call takes by its sizes and layout
alone, each against the formula in 64 bits."""
import pytest
import torch

import moe_reference as ref
from lossless_exponent_reuse_gb300 import ciera, experts
from test_moe_experts_gpu import GROUPS, make, sums, weights
from test_moe_rows_gpu import rand, strided

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gated_slack(a, e):
    """Of silu(gate) * up where the products `a` are within e: |silu'| <= 1.1, exp
    and the division within 16 ulp."""
    g, u = a.chunk(2, 1)
    eg, eu = e.chunk(2, 1)
    return (1.1 * eg * (u.abs() + eu) + ref.silu(g).abs() * eu
            + ref.gated(a).abs() * 16 * ref.U_F32)


@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("groups,unused,K,N", GROUPS)
def test_rows_gathered_inside_products_of_any_size(groups, unused, K, N, kind, monkeypatch):
    """Rows picked by the product itself, however many an expert has, with
    indexes outside x among them."""
    monkeypatch.setattr(experts, "_GATHER_ROWS", 1 << 40)
    T = 50
    offsets, R, tokens = make(groups, unused, T=T)
    if R > 2:
        tokens[R // 2] = T
        tokens[R // 3] = -5
    x = rand(T, K, seed=2)
    w = weights(len(groups), 2 * N, K, kind, scale=1.0 / K ** 0.5)
    rows = ref.gather(x, tokens, R)
    a, size = ref.product(rows, w, offsets)
    e = sums(size, K)
    h, pre = experts.mm_gated(strided(x, kind), w, offsets, tokens=tokens, keep=True)
    ref.within(pre, a, e, "pre")
    ref.within(h, ref.gated(a), gated_slack(a, e), "h")
    ref.within(experts.mm(strided(x, kind), w, offsets, tokens=tokens), a, e, "y")
    assert (h[int(offsets[-1]):] == 0).all() and (pre[int(offsets[-1]):] == 0).all()

    x8, xs = experts.quantize_rows(x)
    w8, ws = experts.quantize_rows(w.contiguous())
    a, size = ref.product(ref.gather(x8.double() * xs.double()[:, None], tokens, R),
                          w8.double() * ws.double()[..., None], offsets)
    e = sums(size, K + 4)
    h, pre = experts.mm_gated(x8, w8, offsets, tokens=tokens, x_scale=xs, w_scale=ws, keep=True)
    ref.within(pre, a, e, "pre, 8 bits")
    ref.within(h, ref.gated(a), gated_slack(a, e), "h, 8 bits")
    y = experts.mm(x8, w8, offsets, tokens=tokens, x_scale=xs, w_scale=ws)
    ref.within(y, a, e, "y, 8 bits")
    assert experts.status() == ciera.OK


def padded(t, grain):
    """The same rows, a multiple of `grain` elements apart."""
    wide = torch.zeros(*t.shape[:-1], -(-t.shape[-1] // grain) * grain, dtype=t.dtype,
                       device=t.device)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


@pytest.mark.parametrize("K,N", [(1001, 520), (76, 72), (9, 264)])
def test_gathered_rows_of_odd_length_keep_the_fast_products(K, N):
    """Rows that are no whole 16-byte words, padded to them: gathering gives what
    the same rows, picked before, give bit for bit, so the same kernel ran."""
    T = 700
    offsets, R, tokens = make([300, 0, 900, 801], 9, T=T)
    x, w = rand(T, K, seed=31), rand(4, N, K, seed=32, scale=1.0 / K ** 0.5)
    rows = ref.gather(x, tokens, R).to(BF16)
    want, size = ref.product(rows.double(), w, offsets)
    y = experts.mm(padded(x, 8), padded(w, 8), offsets, tokens=tokens)
    ref.within(y, want, sums(size, K), "y")
    assert torch.equal(y, experts.mm(padded(rows, 8), padded(w, 8), offsets))

    x8, xs = experts.quantize_rows(x)
    w8, ws = experts.quantize_rows(w)
    r8, rs = experts.gather_rows(x8, tokens, x_scale=xs)
    scales = dict(w_scale=ws)
    y = experts.mm(padded(x8, 16), padded(w8, 16), offsets, tokens=tokens, x_scale=xs, **scales)
    assert torch.equal(y, experts.mm(padded(r8, 16), padded(w8, 16), offsets, x_scale=rs, **scales))

    dy = rand(R, N, seed=33)
    out = [torch.empty(4, N, K, device="cuda") for _ in range(2)]
    experts.mm_dw(dy, padded(x, 8), offsets, tokens=tokens, out=out[0])
    experts.mm_dw(dy, padded(rows, 8), offsets, out=out[1])
    want, size = ref.product_dw(dy.double(), rows.double(), offsets, N, K)
    ref.within(out[0], want, sums(size, 901), "dw", rounded=ref.U_F32)
    assert torch.equal(*out)


@pytest.mark.parametrize("dtype", [BF16, torch.uint8])
@pytest.mark.parametrize("at,stride", [(0, 16), (0, 48), (0, 19), (3, 32), (16, 64)])
@pytest.mark.parametrize("dim", [1, 7, 16])
def test_gather_rows_strided(dim, at, stride, dtype):
    """What lies between the rows stays."""
    e4m3 = dtype is torch.uint8
    x = torch.randint(0, 100, (11, 16), dtype=torch.uint8, device="cuda").to(dtype)[:, :dim]
    tokens = torch.tensor([3, -1, 10, 11, 0], dtype=torch.int32, device="cuda")
    scale = torch.rand(11, device="cuda")
    got_scale = torch.empty(5, device="cuda")
    flat = torch.full((at + 5 * stride,), 77, dtype=dtype, device="cuda")
    want = flat.clone()
    for r, t in enumerate([3, None, 10, None, 0]):
        row = torch.zeros(dim, dtype=dtype, device="cuda") if t is None else x[t]
        want[at + r * stride:at + r * stride + dim] = row
    size = flat.element_size()
    st = ciera.lib().ciera_gather_rows_strided(
        x.data_ptr(), 16, 11, experts.E4M3 if e4m3 else experts.BF16,
        scale.data_ptr() if e4m3 else None, tokens.data_ptr(), 5, dim,
        flat.data_ptr() + at * size, stride, got_scale.data_ptr() if e4m3 else None,
        torch.cuda.current_stream().cuda_stream)
    assert st == ciera.OK and torch.equal(flat, want)
    if e4m3:
        assert torch.equal(got_scale, torch.stack([scale[3], scale[0] * 0, scale[10],
                                                   scale[0] * 0, scale[0]]))


def test_more_columns_than_a_grid_has_blocks_for():
    """Layouts that the tensor cores' loads refuse, with over 65535 * 64 columns."""
    wide, R = 65535 * 64 + 65, 3
    offsets, _, _ = make([2, 1], 0)
    x, w = rand(R, 1, seed=34), rand(2, wide, 1, seed=35)
    want, size = ref.product(x.double(), w, offsets)
    ref.within(experts.mm(x, w, offsets), want, sums(size, 1), "y")
    dy, w = rand(R, 2, seed=36), rand(2, 2, wide, seed=37)
    want, size = ref.product(dy.double(), w.transpose(1, 2), offsets)
    ref.within(experts.mm_dx(dy, w, offsets), want, sums(size, 2), "dx")
    x = rand(R, wide, seed=38)
    want, size = ref.product_dw(dy, x.double(), offsets, 2, wide)
    ref.within(experts.mm_dw(dy, x, offsets), want, sums(size, R), "dw")


@pytest.mark.parametrize("K,N", [(264, 136), (37, 19)])
@pytest.mark.parametrize("dtype,accumulate", [(BF16, False), (BF16, True), (F32, False),
                                              (F32, True)])
@pytest.mark.parametrize("rows", [[40, 0, 130], [400, 300, 500]])
def test_gradients_of_weights_with_experts_side_by_side(rows, K, N, dtype, accumulate):
    """Each row of the result holds that row of all experts: experts closer than
    an expert is long, and nothing overlaps."""
    offsets, R, _ = make(rows, 0)
    dy, x = rand(R, N, seed=39), rand(R, K, seed=40)
    flat = torch.full((N, 3, K + 8), 3.0, dtype=dtype, device="cuda")
    out = flat[:, :, :K].transpose(0, 1)
    want, size = ref.product_dw(dy.double(), x.double(), offsets, N, K)
    slack = sums(size, max(rows))
    if accumulate:
        want, slack = want + 3.0, slack + (3.0 + size) * ref.U_F32
    experts.mm_dw(dy, x, offsets, out=out, accumulate=accumulate)
    ref.within(out, want, slack, "dw", rounded=ref.U_F32 if dtype is F32 else ref.U_BF16)
    assert (flat[:, :, K:] == 3).all()
    assert experts.status() == ciera.OK


def test_gradients_of_weights_refuse_experts_that_overlap():
    offsets, R, _ = make([4, 3], 0)
    dy, x, flat = rand(R, 5), rand(R, 6), torch.zeros(200, dtype=BF16, device="cuda")
    for strides in ((1, 12, 1), (6, 6, 1), (5, 12, 1), (29, 6, 1), (24, 12, 1), (0, 6, 1)):
        with pytest.raises(ValueError, match="overlap"):
            experts.mm_dw(dy, x, offsets, out=flat.as_strided((2, 5, 6), strides))
    for strides in ((30, 6, 1), (6, 12, 1), (54, 12, 1)):
        experts.mm_dw(dy, x, offsets, out=flat.as_strided((2, 5, 6), strides))


def gates(rows, n, seed):
    """Gates from -120 to 120, with ups and gradients of ordinary size."""
    edge = torch.tensor([-120, -100, -90, -88.5, -88, -87.5, -87, -86, -80, -50, -20, -10, -5, -2,
                         -1.28, -1, -0.1, 0, 0.1, 1, 2, 5, 10, 20, 50, 87, 88, 89, 100, 120.0])
    some = torch.randint(0, len(edge), (rows, n), generator=torch.Generator().manual_seed(seed))
    spread = (rand(rows, n, seed=seed, dtype=F32).cpu() * 0.01 + 1) * edge[some]
    return spread.to(BF16).cuda(), rand(rows, n, seed=seed + 1, scale=30.0)


# exp is within 2 + 1.173 |g| units in the last place of 2^-23 (CUDA's bound for
# __expf), the sum, the reciprocal and the products behind it within 8 together;
# a sigmoid below the smallest normal number, 2^-126, may be 0.
def exp_slack(g):
    return (1.173 * g.abs() + 16) * ref.U_F32


@pytest.mark.parametrize("R", [24, 90])
@pytest.mark.parametrize("kind", ["plain", "odd"])
def test_gated_unit_of_large_gates(R, kind):
    """Rows of one 1, so that the products are the weights themselves."""
    K = n = 64
    g, u = gates(n, K, 41)                       # as weights: feature by column
    w = torch.cat([g, u])[None]
    if kind == "odd":
        w = strided(w[0], "odd")[None]
    at = torch.arange(R, device="cuda") % K
    x = torch.nn.functional.one_hot(at, K).to(BF16)
    offsets = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    h, pre = experts.mm_gated(x, w, offsets, keep=True)
    gd, ud = g.double().T[at], u.double().T[at]
    assert torch.equal(pre.double(), torch.cat([gd, ud], 1))
    want = ref.silu(gd) * ud
    ref.within(h, want, want.abs() * exp_slack(gd) + (gd * ud).abs() * 2.0 ** -126, "h")


@pytest.mark.parametrize("R", [24, 90])
@pytest.mark.parametrize("kind", ["plain", "odd"])
def test_gradient_through_large_gates(R, kind):
    n, k = 64, 72
    g, u = gates(R, k, 43)
    w = rand(1, n, k, seed=45)
    at = torch.arange(R, device="cuda") % n
    dy = torch.nn.functional.one_hot(at, n).to(BF16)
    offsets = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    got = experts.mm_dx(strided(dy, kind), w, offsets, gated=torch.cat([g, u], 1))
    d, gd, ud = w[0].double()[at], g.double(), u.double()
    want = ref.gated_gradient(d, torch.cat([gd, ud], 1))
    s = 1 / (1 + torch.exp(-gd))
    size = torch.cat([(d * ud).abs() * (1 + gd.abs()), (d * gd).abs()], 1)
    both = torch.cat([s, s], 1) * torch.cat([exp_slack(gd)] * 2, 1)
    ref.within(got, want, size * both + size * 2.0 ** -126, "dpre")


def e4m3_in(t, pad, at):
    """e4m3 matrices inside a larger buffer of NaNs: rows `pad` bytes further apart, from
    byte `at` on."""
    *stack, rows, dim = t.shape
    ld = dim + pad
    each = rows * ld + pad
    n = stack[0] if stack else 1
    buf = torch.full((at + n * each,), 0x7F, dtype=torch.uint8, device="cuda")
    strides = (each, ld, 1) if stack else (ld, 1)
    v = buf.as_strided(tuple(t.shape), strides, at)
    v.copy_(t.view(torch.uint8))
    return v.view(torch.float8_e4m3fn)


@pytest.mark.parametrize("pad,at", [(16, 32), (16, 1), (3, 0), (5, 7)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("groups,unused,K,N", [GROUPS[i] for i in (2, 3, 4, 8, 9, 13)])
def test_e4m3_operands_anywhere_in_memory(groups, unused, K, N, gather, pad, at):
    T = 60
    offsets, R, tokens = make(groups, unused, T=T if gather else None)
    x8, xs = experts.quantize_rows(rand(T if gather else R, K, seed=46))
    w8, ws = experts.quantize_rows(rand(len(groups), 2 * N, K, seed=47, scale=1.0 / K ** 0.5))
    rows = ref.gather(x8.double() * xs.double()[:, None], tokens, R)
    a, size = ref.product(rows, w8.double() * ws.double()[..., None], offsets)
    e = sums(size, K + 4)
    scales = dict(tokens=tokens, x_scale=xs, w_scale=ws)
    x, w = e4m3_in(x8, pad, at), e4m3_in(w8, pad, at)
    ref.within(experts.mm(x, w, offsets, **scales), a, e, "y")
    h, pre = experts.mm_gated(x, w, offsets, keep=True, **scales)
    ref.within(pre, a, e, "pre")
    ref.within(h, ref.gated(a), gated_slack(a, e), "h")
    assert experts.status() == ciera.OK
