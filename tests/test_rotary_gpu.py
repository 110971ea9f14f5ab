"""Rotary positions, keys and values into their pages, and the pages of a step,
against their definitions."""
import math

import pytest
import torch

import attention_reference as ref
from attention_reference import BF16, E4M3, I32, ints, rand
from lossless_exponent_reuse_gb300 import attention
from moe_reference import within

pytestmark = pytest.mark.gpu
FAR = [0, 1, 2, 100, 4095, 131071, 2 ** 31 - 1, -1, -77777]


def positions_of(T):
    return ints([FAR[t % len(FAR)] if t < 2 * len(FAR) else t for t in range(T)])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,part", [(128, 128), (128, 64), (64, 64), (80, 80), (80, 40), (96, 48),
                                      (96, 24), (256, 256), (1024, 1024), (7, 6), (33, 2), (20, 8),
                                      (128, 0), (2, 2), (1, 0)])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (3, 5), (41, 16)])
def test_rotary_and_its_gradient(tokens, heads, dim, part, interleaved):
    r = attention.rotary_table(part, interleaved=interleaved, amplitude=1.25)
    x, at = rand(tokens, heads, dim, seed=dim + part, scale=3.0), positions_of(tokens)
    for call, sign in ((attention.rotary, 1), (attention.rotary_backward, -1)):
        got = call(x, at, r)
        want, slack = ref.rotary(x, at, r, sign)
        within(got.cpu(), want, slack, (call.__name__, dim, part))
        assert torch.equal(got[..., part:], x[..., part:])


def test_many_tokens():
    for heads, dim in ((32, 128), (7, 80), (1, 64)):
        r = attention.rotary_table(dim)
        x, at = rand(3000, heads, dim), positions_of(3000)
        got = attention.rotary(x, at, r)
        pick = torch.tensor([0, 1, 5, 1499, 2998, 2999], device="cuda")
        want, slack = ref.rotary(x[pick], at[pick], r)
        within(got[pick].cpu(), want, slack)
        # rows one by one give the same
        assert torch.equal(got[1234:1235], attention.rotary(x[1234:1235], at[1234:1235], r))


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(interleaved):
    """d(w . y) / dx by the operator, and by moving single values of x by a power of
    two, which bf16 holds: y's roundings are 2^-8 |y| each, over the step."""
    r = attention.rotary_table(32, interleaved=interleaved, amplitude=0.5)
    x = torch.zeros(2, 1, 40, device="cuda", dtype=BF16)
    w, at = rand(2, 1, 40, seed=3), ints([5, 90])
    dx = attention.rotary_backward(w, at, r).double()
    for i in (0, 1, 15, 16, 31, 32, 39):
        up, down = x.clone(), x.clone()
        up[..., i], down[..., i] = 1.0, -1.0
        y = [attention.rotary(v, at, r).double() for v in (up, down)]
        slope = ((y[0] - y[1]) * w.double()).sum((1, 2)) / 2
        room = (w.double().abs() * y[0].abs()).sum((1, 2)) * 2.0 ** -8
        assert ((slope - dx[:, 0, i]).abs() <= room + 2.0 ** -8 * dx[:, 0, i].abs() + 1e-6).all(), i


def test_gradient_turns_back():
    r = attention.rotary_table(128, scaling="parts", factor=4.0, original=64, amplitude=1.0)
    x, at = rand(50, 4, 128), positions_of(50)
    back = attention.rotary_backward(attention.rotary(x, at, r), at, r)
    # y is rounded once (2^-8 of each value of a pair), turning back mixes the two,
    # and the result is rounded again
    size = torch.hypot(x[..., :64].float(), x[..., 64:].float()).repeat(1, 1, 2)
    assert ((back.float() - x.float()).abs() <= 3 * 2.0 ** -8 * size + 1e-6).all()


@pytest.mark.parametrize("how", ["in place", "view", "odd view", "strided out", "head strides"])
def test_rotary_layouts(how):
    x, at, r = rand(30, 6, 128), positions_of(30), attention.rotary_table(128)
    want = attention.rotary(x, at, r)
    if how == "in place":
        assert attention.rotary(x, at, r, out=x) is x and torch.equal(x, want)
        return
    if how in ("view", "odd view"):
        off = 8 if how == "view" else 1
        wide = torch.full((30, 9, 128 + 16), math.nan, device="cuda", dtype=BF16)
        v = wide[:, 2:8, off:off + 128]
        v.copy_(x)
        assert torch.equal(attention.rotary(v, at, r), want)
        attention.rotary(v, at, r, out=v)
        assert torch.equal(v, want) and torch.isnan(wide[:, :2]).all() and torch.isnan(wide[:, 8]).all()
        assert torch.isnan(wide[..., :off]).all() and torch.isnan(wide[..., off + 128:]).all()
    if how == "strided out":
        wide = torch.full((30, 12, 128), math.nan, device="cuda", dtype=BF16)
        attention.rotary(x, at, r, out=wide[:, 3:9])
        assert torch.equal(wide[:, 3:9], want) and torch.isnan(wide[:, 9:]).all()
    if how == "head strides":
        heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)
        assert torch.equal(attention.rotary(heads_first, at, r), want)


def test_infinities_stay_in_their_pairs():
    x, at, r = rand(4, 2, 64), ints([0, 1, 2, 3]), attention.rotary_table(64)
    clean = attention.rotary(x, at, r)
    x[1, 0, 5], x[2, 1, 40] = math.inf, math.nan
    got = attention.rotary(x, at, r)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[1, 0, [5, 37]] = True
    hit[2, 1, [8, 40]] = True
    assert torch.equal(got[~hit], clean[~hit]) and not torch.isfinite(got[hit]).any()


# ---- keys and values into their pages ----------------------------------------

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("by_head", [False, True])
@pytest.mark.parametrize("dim,part,interleaved", [(128, 128, False), (128, 64, True), (80, 40, False),
                                                  (64, 64, True), (96, 96, False), (40, 10, False),
                                                  (256, 256, False), (7, 4, False), (128, 0, False)])
@pytest.mark.parametrize("tokens,q_heads,heads", [(1, 16, 16), (33, 8, 2), (150, 3, 1)])
def test_append(tokens, q_heads, heads, dim, part, interleaved, by_head, e4m3):
    page, pages = 8, 40
    qkv = rand(tokens, q_heads + 2 * heads, dim, seed=dim + tokens)
    qkv[:, q_heads:] *= torch.exp2(torch.arange(tokens, device="cuda").remainder(9) - 4.0
                                   )[:, None, None].to(BF16)
    q, k, v = qkv.split([q_heads, heads, heads], 1)
    r = attention.rotary_table(part, interleaved=interleaved, amplitude=1.5)
    at = positions_of(tokens)
    shape = (pages, heads, page, dim) if by_head else (pages, page, heads, dim)
    old = [rand(*shape, seed=5 + i) for i in (0, 1)]
    sides = [o.to(E4M3 if e4m3 else BF16) for o in old]
    if by_head:
        sides = [s.transpose(1, 2) for s in sides]
    marks = [torch.full((pages, page, heads), 9, dtype=torch.uint8, device="cuda")
             for _ in range(2)] if e4m3 else []
    cache = attention.Cache(*sides, *marks)
    before = [ref.values(s, None).clone() for s in sides]
    g = torch.Generator().manual_seed(tokens)
    slots = torch.randperm(pages * page, generator=g)[:tokens].to(I32)
    slots[::7] = -1 if tokens > 1 else slots[0]
    if tokens > 20:
        slots[5], slots[6] = pages * page, 2 ** 31 - 1
    got = attention.append(q, k, v, at, slots.cuda(), r, cache)
    want, slack = ref.rotary(q, at, r)
    within(got.cpu(), want, slack)
    live = ((slots >= 0) & (slots < pages * page)).nonzero()[:, 0]
    place = (slots[live].long() // page, slots[live].long() % page)
    rk, slack_k = ref.rotary(k, at, r)
    for i, (y, room, exponent) in enumerate(((rk, slack_k, ref.exponents(k, r)),
                                             (v.double().cpu(), torch.zeros_like(rk),
                                              ref.exponents(v)))):
        now = ref.values(sides[i], None).cpu()
        if e4m3:
            e = marks[i].cpu()
            assert torch.equal(e[place], exponent[live])
            scale = torch.exp2(exponent[live].double() - 127)[..., None]
            # a rounding to 4 bits, or half a step of the smallest values
            off = (now[place] * scale - y[live]).abs()
            room = room[live] * (1 + 2.0 ** -4) + 2.0 ** -4 * y[live].abs() + 2.0 ** -10 * scale
            assert (off <= room).all()
            e[place] = 9
            assert (e == 9).all()
        else:
            within(now[place], y[live], room[live])
        now[place] = before[i].cpu()[place]
        assert torch.equal(now, before[i].cpu())       # all other rows as they were


def test_append_in_place_and_back_through_attention():
    """Rows that append wrote are what attend reads."""
    tokens, heads, dim = 100, 4, 128
    for e4m3 in (False, True):
        pool = attention.page_pool(20, 1, 20)
        cache = attention.page_cache(20, 16, heads, dim, e4m3=e4m3)
        step = attention.assign_pages(pool, ints([0]), ints([tokens]), tokens, 16)
        q, k, v = (rand(tokens, heads, dim, seed=i) for i in range(3))
        r = attention.rotary_table(dim)
        want_q = attention.rotary(q, step.positions, r)
        assert attention.append(q, k, v, step.positions, step.slots, r, cache, out=q) is q
        assert torch.equal(q, want_q)
        got = attention.attend(q, cache, pool.table, step.offsets, step.context)
        ref.check_attend(got, q, cache, pool.table, step.offsets, step.context)


def test_exponents_of_odd_rows():
    rows = torch.zeros(8, 1, 64, device="cuda", dtype=BF16)
    rows[1, 0, 3] = 448.0
    rows[2, 0, 3] = 450.0
    rows[3, 0, 60] = math.inf
    rows[4, 0, 60] = math.nan
    rows[5, 0, 1] = 2.0 ** -120
    rows[6, 0, 1] = 3.0e38
    rows[7, 0, 1] = -7.0 * 2.0 ** -7
    cache = attention.page_cache(1, 8, 1, 64, e4m3=True)
    r = attention.rotary_table(0)
    attention.append(rows, rows, rows, ints([0] * 8), ints(list(range(8))), r, cache)
    want = ref.exponents(rows)
    assert torch.equal(cache.key_exponent[0].cpu(), want)
    assert torch.equal(cache.value_exponent[0].cpu(), want)
    assert want[:, 0].tolist() == [27, 127, 128, 255, 255, 27, 127 + 119, 127 - 13]
    assert float(cache.value[0, 7, 0, 1].float()) == -448.0


# ---- pages of a step ---------------------------------------------------------

def check_assign(table, free, count, cached, new, tokens, page, width_pad=0):
    rows = [list(row) for row in table]
    want = ref.assign(rows, free, count, cached, new, tokens, page)
    width = len(table[0])
    t = torch.full((len(table), width + width_pad), 55, dtype=I32, device="cuda")
    t[:, :width] = ints(table).view(len(table), width)
    pool = attention.Pool(t[:, :width], ints(free), ints([count]))
    step = attention.assign_pages(pool, ints(cached), ints(new), tokens, page)
    got = (step.offsets, step.context, step.lengths, step.positions, step.slots)
    for name, g, w in zip(("offsets", "context", "lengths", "positions", "slots"), got, want):
        assert g.tolist() == w, (name, cached, new, tokens, page)
    assert int(step.pool.count) == want[5] and int(pool.count) == count
    assert step.pool.table.tolist() == rows and (t[:, width:] == 55).all()
    return step


def setup(R, width, page, seed, most_cached, most_new):
    g = torch.Generator().manual_seed(seed)
    cached = torch.randint(0, most_cached + 1, (R,), generator=g).tolist()
    new = torch.randint(0, most_new + 1, (R,), generator=g).tolist()
    pages = sum(-(-c // page) for c in cached)
    order = torch.randperm(pages + 500, generator=g).tolist()
    table = []
    for c in cached:
        held = -(-c // page)
        table.append([order.pop() for _ in range(held)] + [-1] * (width - held))
    return table, order, cached, new


@pytest.mark.parametrize("R", [1, 2, 31, 33, 200, 1025, 2500])
@pytest.mark.parametrize("page", [1, 16, 20])
def test_assign_pages(R, page):
    table, free, cached, new = setup(R, 80 // page + 3, page, R + page, 50, 20)
    total = sum(new)
    for count in (len(free), 0, min(len(free), 7), min(len(free), 100)):
        check_assign(table, free, count, cached, new, total, page, width_pad=3)
    check_assign(table, free, len(free), cached, new, total + 9, page)
    check_assign(table, free, len(free), cached, new, max(total - 5, 0), page)


def test_assign_long_prompts():
    table = [[-1] * 700, [-1] * 700]
    free = list(range(1400))
    check_assign(table, free, 1400, [0, 0], [9999, 1200], 11199, 16)
    check_assign(table, free, 1400, [0, 0], [12000, 1200], 13200, 16)    # past the table


def test_assign_odd_lengths():
    table = [[3, -1], [-1, -1], [-1, -1], [4, 5]]
    free = [0, 1, 2]
    check_assign(table, free, 3, [5, -4, 0, 16], [0, 3, -7, 0], 10, 8)
    check_assign(table, free, 3, [16, 2 ** 31 - 1, 0, 9], [1, 2 ** 31 - 1, 1, 1], 10, 8)
    step = check_assign([[-1]], [7], 1, [0], [0], 0, 8)
    assert step.positions.numel() == 0
    assert check_assign([[-1]], [0], 1, [0], [1], 1, 2 ** 31 - 1).slots.tolist() == [0]
    empty = attention.Pool(torch.empty(0, 4, dtype=I32, device="cuda"), ints([1, 2]), ints([2]))
    got = attention.assign_pages(empty, ints([]), ints([]), 3, 16)
    assert got.offsets.tolist() == [0] and got.slots.tolist() == [-1] * 3 and int(got.pool.count) == 2


def test_a_pool_from_step_to_step():
    """Requests come, grow, starve, leave, and come again: no page is ever held twice."""
    page, width, pages = 4, 12, 40
    pool = attention.page_pool(pages, 6, width)
    lengths = ints([0] * 6)
    g = torch.Generator().manual_seed(1)
    for turn in range(40):
        new = torch.randint(0, 9, (6,), generator=g)
        step = attention.assign_pages(pool, lengths, new.to(I32).cuda(), int(new.sum()), page,
                                      count=pool.count)
        lengths = step.lengths
        if turn % 3 == 2:
            done = torch.rand(6, generator=g) < 0.4
            held = lengths.clone()
            out = attention.release_pages(pool, lengths, done.cuda(), page, count=pool.count)
            assert out.count is pool.count
            assert lengths.tolist() == [0 if d else n for d, n in zip(done.tolist(), held.tolist())]
        rows, n = pool.table.tolist(), lengths.tolist()
        used = [p for row in rows for p in row if p >= 0]
        assert all(sum(p >= 0 for p in row) == -(-k // page) for row, k in zip(rows, n))
        free = pool.free.tolist()[:int(pool.count)]
        assert sorted(used + free) == list(range(pages))


def test_release_order_and_odd_entries():
    table = ints([[3, -1, 9], [7, 8, -1], [100, 2, 5], [1, 4, 6]])
    free = ints([50, 51] + [0] * 10)
    pool = attention.Pool(table, free, ints([2]))
    lengths = ints([9, 5, 30, 12])
    out = attention.release_pages(pool, lengths, torch.tensor([1, 0, 1, 1], dtype=torch.uint8,
                                                              device="cuda"), 4)
    assert int(out.count) == 9 and int(pool.count) == 2
    assert free.tolist()[:9] == [50, 51, 3, 9, 2, 5, 1, 4, 6]
    assert table.tolist() == [[-1] * 3, [7, 8, -1], [-1] * 3, [-1] * 3]
    assert lengths.tolist() == [0, 5, 0, 0]
