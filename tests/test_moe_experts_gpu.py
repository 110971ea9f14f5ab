"""Products grouped by expert against their formulas in 64 bits: ragged and
empty groups, rows past the last group, gathered rows, views of a bucket,
sizes and alignments that do and do not suit the tensor cores."""
import pytest
import torch

import moe_reference as ref
from lossless_exponent_reuse_gb300 import ciera, experts
from test_moe_rows_gpu import rand, strided

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

# groups, in rows each; unused rows at the end; columns in and out
GROUPS = [
    ([1], 0, 64, 64),
    ([0, 0, 3], 0, 64, 32),
    ([1, 0, 1, 1, 0, 1, 1, 1], 0, 2048, 128),
    ([5, 0, 17, 130], 9, 136, 264),
    ([300, 1, 0, 0, 64, 128, 127, 129], 40, 512, 192),
    ([0, 0, 0], 7, 128, 64),
    ([33] * 16, 0, 264, 520),
    ([700, 2], 3, 72, 40),
    ([3, 40, 20], 2, 37, 19),            # rows the tensor cores cannot load
    ([260, 250], 0, 1000, 1001),
    ([4] * 130, 5, 128, 136),
    ([16, 31, 32, 33, 15, 1, 48, 0, 80], 0, 320, 384),
    ([1, 2, 3, 4], 6, 4096, 1000),
    ([37 * i % 611 for i in range(24)], 50, 520, 1544),   # several tiles for every pair of blocks
    ([29 * i % 64 for i in range(100)], 3, 264, 2056),    # and for every single block
]


def test_large_cases_fill_the_device_several_times():
    """The two cases above that are meant to: tiles of 256 x 256, and of 128 x 64."""
    pairs = sum(-(-n // 256) for n in GROUPS[-2][0]) * -(-GROUPS[-2][3] // 256)
    single = sum(-(-n // 64) for n in GROUPS[-1][0]) * -(-GROUPS[-1][3] // 128)
    assert pairs > 3 * 76 and single > 3 * 152
    assert sum(GROUPS[-2][0]) > 32 * 24 and sum(GROUPS[-1][0]) <= 32 * 100


def make(groups, unused, seed=0, T=None):
    counts = torch.tensor(groups)
    offsets = torch.zeros(len(groups) + 1, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    R = int(offsets[-1]) + unused
    tokens = None
    if T is not None:
        g = torch.Generator().manual_seed(seed)
        tokens = torch.randint(0, T, (R,), generator=g, dtype=torch.int32)
        tokens[int(offsets[-1]):] = -1
        tokens = tokens.cuda()
    return offsets.cuda(), R, tokens


def weights(E, N, K, kind, seed=0, scale=0.1):
    w = rand(E, N, K, seed=seed, scale=scale)
    if kind == "plain":
        return w
    # inside a larger buffer: experts and rows further apart, at an odd or even place
    pad, at = (8, 16) if kind == "wide" else (3, 1)
    ld = K + pad
    buf = torch.full((at + E * (N * ld + pad),), float("nan"), dtype=BF16, device="cuda")
    v = buf.as_strided((E, N, K), (N * ld + pad, ld, 1), at)
    v.copy_(w)
    return v


def sums(size, terms):
    return size * (terms + 2) * ref.U_F32


@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("groups,unused,K,N", GROUPS)
def test_forward(groups, unused, K, N, kind):
    offsets, R, _ = make(groups, unused)
    x = rand(R, K, seed=1)
    x[int(offsets[-1]):] = float("nan")                 # unused rows are not read
    w = weights(len(groups), N, K, kind)
    want, size = ref.product(torch.nan_to_num(x.double()), w, offsets)
    y = experts.mm(strided(x, kind), w, offsets)
    ref.within(y, want, sums(size, K), "y")
    assert (y[int(offsets[-1]):] == 0).all()
    assert experts.status() == ciera.OK


@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("groups,unused,K,N", GROUPS)
def test_forward_gated_and_gathered(groups, unused, K, N, kind):
    T = 50
    offsets, R, tokens = make(groups, unused, T=T)
    x = rand(T, K, seed=2)
    w = weights(len(groups), 2 * N, K, kind, scale=1.0 / K ** 0.5)
    a, size = ref.product(ref.gather(x, tokens, R), w, offsets)
    h, pre = experts.mm_gated(strided(x, kind), w, offsets, tokens=tokens, keep=True)
    e = sums(size, K)
    ref.within(pre, a, e, "pre")
    # |silu'| <= 1.1, exp and the division within 8 ulp
    want = ref.gated(a)
    g, u = a.chunk(2, 1)
    eg, eu = e.chunk(2, 1)
    slack = 1.1 * eg * (u.abs() + eu) + ref.silu(g).abs() * eu + want.abs() * 16 * ref.U_F32
    ref.within(h, want, slack, "h")
    assert torch.equal(h, experts.mm_gated(strided(x, kind), w, offsets, tokens=tokens))
    assert (h[int(offsets[-1]):] == 0).all() and (pre[int(offsets[-1]):] == 0).all()
    assert experts.status() == ciera.OK


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("groups,unused,K,N", GROUPS)
def test_forward_e4m3(groups, unused, K, N, gather):
    T = 40
    offsets, R, tokens = make(groups, unused, T=T if gather else None)
    x8, xs = experts.quantize_rows(rand(T if gather else R, K, seed=3))
    for gated in (False, True):
        w8, ws = experts.quantize_rows(rand(len(groups), 2 * N if gated else N, K, seed=4,
                                            scale=1.0 / K ** 0.5))
        rows = ref.gather(x8.double() * xs.double()[:, None], tokens, R)
        a, size = ref.product(rows, w8.double() * ws.double()[..., None], offsets)
        e = sums(size, K + 4)
        if not gated:
            y = experts.mm(x8, w8, offsets, tokens=tokens, x_scale=xs, w_scale=ws)
            ref.within(y, a, e, "y")
        else:
            h, pre = experts.mm_gated(x8, w8, offsets, tokens=tokens, x_scale=xs, w_scale=ws,
                                      keep=True)
            ref.within(pre, a, e, "pre")
            g, u = a.chunk(2, 1)
            eg, eu = e.chunk(2, 1)
            want = ref.gated(a)
            slack = 1.1 * eg * (u.abs() + eu) + ref.silu(g).abs() * eu \
                + want.abs() * 16 * ref.U_F32
            ref.within(h, want, slack, "h")
    assert experts.status() == ciera.OK


@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("groups,unused,K,N", GROUPS)
def test_gradient_of_rows(groups, unused, K, N, kind):
    offsets, R, _ = make(groups, unused)
    dy = rand(R, N, seed=5)
    dy[int(offsets[-1]):] = float("nan")
    w = weights(len(groups), N, K, kind)
    want, size = ref.product(torch.nan_to_num(dy.double()), w.transpose(1, 2), offsets)
    dx = experts.mm_dx(strided(dy, kind), w, offsets)
    ref.within(dx, want, sums(size, N), "dx")
    pre = rand(R, 2 * K, seed=6, scale=2.0)
    pre[int(offsets[-1]):] = float("nan")
    got = experts.mm_dx(strided(dy, kind), w, offsets, gated=pre)
    pre = torch.nan_to_num(pre.double())
    factor = ref.gated_gradient(torch.ones_like(want), pre)
    slack = (torch.cat([sums(size, N)] * 2, 1) * factor.abs()
             + ref.gated_gradient(want.abs(), pre.abs()).abs() * 32 * ref.U_F32)
    ref.within(got, ref.gated_gradient(want, pre), slack, "dpre")
    assert (dx[int(offsets[-1]):] == 0).all() and (got[int(offsets[-1]):] == 0).all()
    assert experts.status() == ciera.OK


@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("groups,unused,K,N", GROUPS)
def test_gradient_of_weights(groups, unused, K, N, gather, kind):
    T, E = 45, len(groups)
    offsets, R, tokens = make(groups, unused, T=T if gather else None)
    dy = rand(R, N, seed=7)
    x = rand(T if gather else R, K, seed=8)
    used = int(offsets[-1])
    dy[used:] = float("nan")
    if not gather:
        x[used:] = float("nan")
    want, size = ref.product_dw(torch.nan_to_num(dy.double()),
                                torch.nan_to_num(ref.gather(x, tokens, R)), offsets, N, K)
    deep = sums(size, max(groups))
    dw = experts.mm_dw(strided(dy, kind), strided(x, kind), offsets, tokens=tokens)
    ref.within(dw, want, deep, "dw")
    out = torch.empty(E, N, K, device="cuda")
    assert experts.mm_dw(dy, x, offsets, tokens=tokens, out=out) is out
    ref.within(out, want, deep, "dw float", rounded=ref.U_F32)
    # added to what a strided buffer holds
    for dtype in (F32, BF16):
        base = rand(E, N, K, seed=9, dtype=dtype)
        acc = torch.zeros(E, N + 1, K + 5, dtype=dtype, device="cuda")[:, :N, :K]
        acc.copy_(base)
        experts.mm_dw(dy, x, offsets, tokens=tokens, out=acc, accumulate=True)
        ref.within(acc, base.double() + want, deep + (base.double().abs() + size) * ref.U_F32,
                   "accumulated", rounded=ref.U_F32 if dtype == F32 else ref.U_BF16)
        for e, n in enumerate(groups):
            if n == 0:
                assert torch.equal(acc[e], base[e])
    assert experts.status() == ciera.OK


@pytest.mark.parametrize("groups", [[1, 0, 40], [250, 270, 248], [255, 256, 257],
                                    [260, 300, 209], [700, 0, 130]])
@pytest.mark.parametrize("K,N", [(272, 40), (264, 272), (8, 8), (520, 304)])
def test_gradient_of_weights_from_few_and_from_many_rows(groups, K, N):
    """On both sides of 256 rows an expert, with last tiles of few features and
    few rows, into a strided buffer whose gaps stay."""
    offsets, R, _ = make(groups, 0)
    dy, x = rand(R, N, seed=21), rand(R, K, seed=22)
    want, size = ref.product_dw(dy.double(), x.double(), offsets, N, K)
    flat = torch.full((3, N + 2, K + 8), 7.0, dtype=BF16, device="cuda")
    out = flat[:, 1:N + 1, :K]
    experts.mm_dw(dy, x, offsets, out=out)
    ref.within(out, want, sums(size, max(groups)), "dw")
    assert (flat[:, 0] == 7).all() and (flat[:, N + 1] == 7).all() and (flat[:, :, K:] == 7).all()
    assert experts.status() == ciera.OK


def test_a_group_with_infinities_does_not_touch_its_neighbours():
    groups, K, N = [20, 1, 50, 7], 192, 136
    offsets, R, _ = make(groups, 3)
    x, dy, w = rand(R, K, seed=10), rand(R, N, seed=11), weights(4, N, K, "plain")
    x[20] = float("inf")
    dy[20] = float("nan")
    y = experts.mm(x, w, offsets)
    dw = experts.mm_dw(dy, x, offsets)
    dx = experts.mm_dx(dy, w, offsets)
    keep = [i for i in range(R) if i != 20]
    assert torch.isfinite(y[keep]).all() and torch.isfinite(dx[keep]).all()
    assert torch.isfinite(dw[[0, 2, 3]]).all()


def test_offsets_and_tokens_outside_are_taken_for_the_nearest_or_none():
    K, N = 128, 64
    x, w = rand(20, K, seed=12), weights(3, N, K, "plain")
    offsets = torch.tensor([0, 9, 4, 99], dtype=torch.int32, device="cuda")   # 0, 9, 9, 20
    want, size = ref.product(x.double(), w, offsets)
    ref.within(experts.mm(x, w, offsets), want, sums(size, K), "y")
    tokens = torch.arange(20, dtype=torch.int32, device="cuda")
    tokens[[2, 15]] = torch.tensor([-7, 20], dtype=torch.int32, device="cuda")
    y = experts.mm(x, w, offsets, tokens=tokens)
    assert (y[2] == 0).all() and (y[15] == 0).all()
    dw = experts.mm_dw(rand(20, N, seed=13), x, offsets, tokens=tokens)
    rows = ref.gather(x, tokens, 20)
    want, size = ref.product_dw(rand(20, N, seed=13), rows, offsets, N, K)
    ref.within(dw, want, sums(size, 20), "dw")


def test_no_rows_and_no_experts():
    w = weights(2, 16, 24, "plain")
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert experts.mm(rand(0, 24), w, offsets).shape == (0, 16)
    assert experts.mm_dx(rand(0, 16), w, offsets).shape == (0, 24)
    assert (experts.mm_dw(rand(0, 16), rand(0, 24), offsets) == 0).all()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = experts.mm(rand(5, 24), w[:0], none)
    assert (y == 0).all()


def test_gradients_against_differences():
    groups, K, N = [6, 0, 11], 64, 48
    offsets, R, _ = make(groups, 0)
    x, w, d = rand(R, K, seed=14), weights(3, 2 * N, K, "plain"), rand(R, N, seed=15)

    def loss(xv, wv):
        return (ref.gated(ref.product(xv, wv, offsets)[0]) * d.double()).sum()

    _, pre = experts.mm_gated(x, w, offsets, keep=True)
    eye = torch.eye(N, dtype=BF16, device="cuda").expand(3, N, N)
    dpre = experts.mm_dx(d, eye, offsets, gated=pre)   # down = identity: dh = d
    dx = experts.mm_dx(dpre, w, offsets)
    dw = experts.mm_dw(dpre, x, offsets, out=torch.empty(3, 2 * N, K, device="cuda"))
    step = 1e-4
    vx, vw = rand(R, K, seed=16).double(), rand(3, 2 * N, K, seed=17).double()
    xd, wd = x.double(), w.double()
    for got, v, slope in (
            (dx, vx, loss(xd + step * vx, wd) - loss(xd - step * vx, wd)),
            (dw, vw, loss(xd, wd + step * vw) - loss(xd, wd - step * vw))):
        # pre, dpre and dx are each within 2^-8: at most 4 * 2^-8 of the terms' sizes
        size = (got.double().abs() * v.abs()).sum()
        assert abs((got.double() * v).sum() - slope / (2 * step)) <= 4 * 2.0 ** -8 * size


def test_strides_past_32_bits():
    """Experts' weights more than 2^32 bytes apart."""
    K, N, far = 64, 32, (1 << 31) + 64
    buf = torch.empty(far + N * K, dtype=BF16, device="cuda")
    w = buf.as_strided((2, N, K), (far, K, 1))
    w.copy_(rand(2, N, K, seed=18, scale=0.1))
    offsets, R, _ = make([5, 40], 0)
    x, dy = rand(R, K, seed=19), rand(R, N, seed=20)
    want, size = ref.product(x.double(), w, offsets)
    ref.within(experts.mm(x, w, offsets), want, sums(size, K), "y")
    want, size = ref.product(dy.double(), w.transpose(1, 2), offsets)
    ref.within(experts.mm_dx(dy, w, offsets), want, sums(size, N), "dx")
    want, size = ref.product_dw(dy, x.double(), offsets, N, K)
    experts.mm_dw(dy, x, offsets, out=w)
    ref.within(w, want, sums(size, 40), "dw")


def test_captured_in_a_graph():
    groups, K, N = [40, 3, 0, 90], 256, 128
    offsets, R, _ = make(groups, 0)
    x, w = rand(R, K, seed=21), weights(4, 2 * N, K, "plain")
    want = experts.mm_gated(x, w, offsets)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        experts.mm_gated(x, w, offsets)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        h = experts.mm_gated(x, w, offsets)
    h.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want)
