"""Attention over pages at its edges: values out of a row's sight and what looking at
them costs, rows and powers of two of any magnitude, tiles longer than a wait's limit,
8-bit pages behind 32 bits."""
import math

import pytest
import torch

import attention_reference as ref
from attention_reference import BF16, ints, rand
from lossless_exponent_reuse_gb300 import attention, ciera, experts
from test_attention_gpu import batch

pytestmark = pytest.mark.gpu


def places(table, page, keys):
    keys = torch.as_tensor(keys, device="cuda")
    return table[0].long()[keys // page], keys % page


def put(cache, slot, head, d, bad):
    """``bad`` in the values of some keys; of 8 bits NaN by value, or by exponent where d
    is None."""
    if cache.value_exponent is None:
        cache.value[(*slot, head, slice(None) if d is None else d)] = bad
    elif d is None:
        cache.value_exponent[(*slot, head)] = 255
    else:
        cache.value.view(torch.uint8)[(*slot, head, d)] = 0xFF


# tokens, page, size of a head, query heads to two: rows by tcgen05, by few rows, one by one
FORMS = [(300, 16, 128, 2), (140, 24, 64, 6), (300, 20, 80, 4), (7, 16, 128, 4), (9, 20, 256, 2),
         (12, 1, 64, 4), (12, 16, 66, 2)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new,page,dim,q_heads", FORMS)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_in_sight_and_out_of_it(new, page, dim, q_heads, bad, e4m3):
    """The same place of the head and another one, NaN or infinite for all rows, for the
    last ones, for every key: each row has what it sees, no more and no less."""
    if e4m3 and bad == math.inf:
        pytest.skip("e4m3 has no infinity")
    cached = 190
    L = cached + new
    last = [L - 1, L - 2, L - 5]
    cases = [
        [([0], 3, bad)],                                     # all see it
        [([0], 3, bad), (last, 3, bad)],                     # and more of it out of sight
        [([0], 3, bad), (last, 5, bad)],                     # another place out of sight
        [([L - new // 2], dim - 1, bad), ([0], 0, bad)],
        [(range(L), 7, bad)],                                # in every key
        [(range(L), 7, bad), (last, 8, bad)],
        [(range(cached, L, 3), 2, bad)],
        [([L - 1], None, bad)],                              # a whole row
    ]
    for marks in cases:
        q, cache, table, offsets, context = batch([new], [cached], q_heads, 2, dim, page, e4m3=e4m3)
        for keys, d, value in marks:
            put(cache, places(table, page, list(keys)), 1, d, value)
        got = attention.attend(q, cache, table, offsets, context)
        ref.check_attend(got, q, cache, table, offsets, context, what=marks)
        assert torch.isfinite(got[:, :q_heads // 2]).all()
    assert experts.status() == ciera.OK


def microseconds(fn, n=5):
    fn()
    best = math.inf
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(n):
            fn()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / n * 1000)
    return best


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new,cached", [(4096, 0), (512, 8192), (4, 8192)])
def test_a_nan_in_sight_costs_little(new, cached, e4m3):
    """One NaN that every row sees, or one in the same place of every key: no row is
    computed again, which would take some thousand times as long."""
    heads, dim, page = 16, 128, 16
    L = cached + new
    cache, table = ref.paged([L], page, heads, dim, e4m3=e4m3)
    q, off, context = rand(new, heads, dim, seed=3), ints([0, new]), ints([L])
    call = lambda: attention.attend(q, cache, table, off, context)
    clean = microseconds(call)
    put(cache, places(table, page, [0]), slice(None), 0, math.nan)
    assert microseconds(call) < 20 * clean
    got = call()
    assert torch.isnan(got[:, :, 0]).all() and torch.isfinite(got[:, :, 1:]).all()
    put(cache, tuple(x[:, None] for x in places(table, page, range(L))),
        torch.arange(heads, device="cuda"), 1, math.nan)
    assert microseconds(call) < 20 * clean
    got = call()
    assert torch.isnan(got[:, :, :2]).all() and torch.isfinite(got[:, :, 2:]).all()
    assert experts.status() == ciera.OK


@pytest.mark.parametrize("dim,e4m3,page", [(66, False, 16), (129, False, 5), (7, False, 1), (72, True, 16),
                                           (250, True, 20), (33, True, 3)])
def test_rows_one_by_one(dim, e4m3, page):
    """Heads that no other form takes: lengths around the keys of a step, pages that are
    not there, queries and keys that are infinite or NaN."""
    lengths = [1, 31, 32, 33, 63, 64, 65, 100]
    new = [1, 3, 1, 33, 1, 2, 1, 40]
    args = [new, [n - k for n, k in zip(lengths, new)], 4, 2, dim, page]
    q, cache, table, off, context = batch(*args, e4m3=e4m3)
    got = attention.attend(q, cache, table, off, context)
    ref.check_attend(got, q, cache, table, off, context, what=(dim, e4m3, page))
    table[7, 1], table[3, 0] = -1, cache.key.shape[0]
    got = attention.attend(q, cache, table, off, context)
    ref.check_attend(got, q, cache, table, off, context, what=(dim, e4m3, page))
    clean = got.clone()
    # scores of plus and minus infinity, and of NaN, in rows of their own
    last, first = int(off[-1]) - 1, int(off[3])
    q[last, 0, -1], q[last - 1, 3, 0], q[first, 2] = math.inf, -math.inf, math.nan
    if e4m3:
        cache.key_exponent[table[6, 0].long(), 0, 1] = 255
    else:
        cache.key[table[6, 0].long(), 0, 1, 0] = math.nan
    got = attention.attend(q, cache, table, off, context)
    row = int(off[6])
    odd = torch.zeros_like(got, dtype=torch.bool)
    odd[last, 0] = odd[last - 1, 3] = odd[first, 2] = odd[row, 2] = odd[row, 3] = True
    assert torch.isnan(got[odd]).all() and torch.equal(got[~odd], clean[~odd])
    assert experts.status() == ciera.OK


@pytest.mark.parametrize("new,page,dim,q_heads", [(1, 16, 128, 4), (3, 20, 64, 4), (5, 16, 256, 2),
                                                  (16, 16, 128, 2), (150, 16, 128, 4), (4, 16, 72, 2)])
@pytest.mark.parametrize("q_power,k_power", [(124, -124), (100, -100), (40, -40), (-60, 60), (-100, 100),
                                             (-113, 113), (-119, 119), (-124, 119)])
def test_queries_of_any_magnitude(new, page, dim, q_heads, q_power, k_power):
    """8-bit keys whose powers of two make up for the queries': every form has the same
    scores, and rows of other magnitudes beside them their own."""
    L, heads = new + 150, 2
    rows = lambda kind, r, n: rand(n, heads, dim, seed=70 + kind, dtype=torch.float32) / 64
    cache, table = ref.paged([L], page, heads, dim, e4m3=True, value=rows)
    slot = places(table, page, range(L))
    cache.key_exponent[slot] = 127 + k_power
    q = (rand(new, q_heads, dim, seed=5, dtype=torch.float64).clamp(-3, 3) * 2.0 ** q_power).to(BF16)
    q[0, 0, :3] *= 2.0 ** -7               # within a row too
    q[0, 1] = 0
    off, context = ints([0, new]), ints([L])
    for scale in (None, 4.0, -4.0):
        got = attention.attend(q, cache, table, off, context, scale=scale)
        ref.check_attend(got, q, cache, table, off, context, scale, what=(new, dim, q_power))
    # a value that is infinite, among large and small ones: every score minus infinity
    key = cache.key.view(torch.uint8)
    key[(*slot, 0, 0)] = 0x38
    q[0, 0, 0] = -math.inf
    got = attention.attend(q, cache, table, off, context)
    assert (got[0, 0] == 0).all() and torch.isfinite(got).all()
    assert experts.status() == ciera.OK


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_tile_longer_than_the_limit(e4m3):
    """Tiles of a million keys take a block some 12 ms each: with a limit of 2 ms no wait runs
    out, as every unit's loads and products go on."""
    page, dim, L = 128, 128, 1 << 20
    cache = attention.page_cache(1, page, 1, dim, e4m3=e4m3)
    v = rand(dim, seed=1).to(torch.float8_e4m3fn).to(BF16)
    cache.value.view(torch.uint8 if e4m3 else BF16)[:] = (
        v.to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else v)
    if e4m3:
        cache.key_exponent.fill_(127), cache.value_exponent.fill_(127)
    table = torch.zeros(2, L // page, dtype=torch.int32, device="cuda")
    new = [320 * 256, 100]
    q, off = rand(sum(new), 1, dim, seed=2), ints([0, new[0], sum(new)])
    try:
        ciera.set_wait_timeout_ns(2 * 10 ** 6)
        got = attention.attend(q, cache, table, off, ints([L, L]))
        assert experts.status() == ciera.OK
    finally:
        ciera.set_wait_timeout_ns(10 ** 9)
    # keys of zeros: the mean of values that are all the same
    assert torch.equal(got, v.expand_as(got))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("by_head", [False, True])
def test_append_and_attend_behind_32_bits(e4m3, by_head):
    """The last pages of a cache of more than 2^32 values a side, written and read: 8-bit
    rows' bytes and exponents too, and by every form."""
    page, heads, dim = 512, 32, 128
    pages = 2 ** 32 // (page * heads * dim) + 200
    shape = (pages, heads, page, dim) if by_head else (pages, page, heads, dim)
    order = (lambda t: t.transpose(1, 2)) if by_head else (lambda t: t)
    kind = torch.float8_e4m3fn if e4m3 else BF16
    sides = [order(torch.empty(shape, dtype=kind, device="cuda")) for _ in range(2)]
    if e4m3:
        # exponents with gaps: places behind 2^31 too
        sides += [order(torch.empty(*shape[:3], 32, dtype=torch.uint8, device="cuda"))[..., 7]
                  for _ in range(2)]
    cache = attention.Cache(*sides)
    assert cache.key.numel() > 2 ** 32
    used = [pages - 1, 5, pages - 2]
    L = 2 * page + 300
    at = torch.arange(L, device="cuda")
    slots = torch.tensor(used, device="cuda")[at // page] * page + at % page
    assert int(slots.max()) * heads * dim > 2 ** 32
    r = attention.rotary_table(dim)
    q, k, v = (rand(L, heads, dim, seed=s, scale=1.5) for s in (1, 2, 3))
    turned = attention.append(q, k, v, at.int(), slots.int(), r, cache)
    small = attention.page_cache(3, page, heads, dim, e4m3=e4m3)
    assert torch.equal(turned, attention.append(q, k, v, at.int(), at.int(), r, small))
    for side, want in zip(cache, small):
        if side is None:
            continue
        got = side.view(torch.uint8) if e4m3 else side
        want = want.view(torch.uint8) if e4m3 else want
        for i, p in enumerate(used):
            n = min(page, L - i * page)
            assert torch.equal(got[p, :n], want[i, :n])
    for new in (1, 3, 130):
        o = attention.attend(turned[L - new:], cache, ints([used]), ints([0, new]), ints([L]))
        assert torch.equal(o, attention.attend(turned[L - new:], small, ints([[0, 1, 2]]),
                                               ints([0, new]), ints([L])))
        if new == 130:
            ref.check_attend(o, turned[L - new:], small, ints([[0, 1, 2]]), ints([0, new]), ints([L]))
    assert experts.status() == ciera.OK


@pytest.mark.parametrize("e4m3", [False, True])
def test_heads_of_odd_size_behind_32_bits(e4m3):
    """The same of the forms for any layout: rows of 72 8-bit values, of 127 of 16 bits."""
    page, heads, dim = 512, 8, 72 if e4m3 else 127
    pages = 2 ** 32 // (page * heads * dim) + 100
    kind = torch.float8_e4m3fn if e4m3 else BF16
    sides = [torch.empty(pages, page, heads, dim, dtype=kind, device="cuda") for _ in range(2)]
    if e4m3:
        sides += [torch.empty(pages, page, heads, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache, used, L = attention.Cache(*sides), [pages - 1, pages - 2], page + 40
    at = torch.arange(L, device="cuda")
    slots = torch.tensor(used, device="cuda")[at // page] * page + at % page
    r = attention.rotary_table(dim - dim % 2)
    q, k, v = (rand(L, heads, dim, seed=s) for s in (1, 2, 3))
    small = attention.page_cache(2, page, heads, dim, e4m3=e4m3)
    turned = attention.append(q, k, v, at.int(), slots.int(), r, cache)
    assert torch.equal(turned, attention.append(q, k, v, at.int(), at.int(), r, small))
    for new in (1, 40):
        o = attention.attend(turned[L - new:], cache, ints([used]), ints([0, new]), ints([L]))
        assert torch.equal(o, attention.attend(turned[L - new:], small, ints([[0, 1]]),
                                               ints([0, new]), ints([L])))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new,page,dim,q_heads", [(300, 16, 128, 4), (290, 20, 64, 6), (14, 16, 128, 2),
                                                  (20, 1, 64, 4), (40, 16, 66, 2)])
def test_rows_that_see_nothing_of_bad_values(new, page, dim, q_heads, e4m3):
    """More new tokens than keys, and values that are NaN among the keys: the first rows see
    none and are zeros, the last ones what they see."""
    L = new // 3
    cache, table = ref.paged([L, 50], page, 2, dim, e4m3=e4m3)
    for key in (L // 2, L - 1):
        put(cache, places(table, page, [key]), 1, 3, math.nan)
    q, off = rand(new + 5, q_heads, dim, seed=6), ints([0, new, new + 5])
    context = ints([L, 50])
    got = attention.attend(q, cache, table, off, context)
    ref.check_attend(got, q, cache, table, off, context)
    assert (got[:new - L] == 0).all() and torch.isnan(got[new - 1, q_heads // 2:, 3]).all()
    assert experts.status() == ciera.OK


@pytest.mark.parametrize("new", [1, 3])
def test_large_queries_over_many_blocks(new):
    """Rows that are computed value by value in parts that several blocks leave, beside rows
    that are not."""
    page, dim, heads, L = 16, 128, 2, 9000
    rows = lambda kind, r, n: rand(n, heads, dim, seed=80 + kind, dtype=torch.float32) / 64
    cache, table = ref.paged([L], page, heads, dim, e4m3=True, value=rows)
    cache.key_exponent[places(table, page, range(L))] = 127 - 120
    q = (rand(new, 4, dim, seed=8, dtype=torch.float64).clamp(-3, 3) * 2.0 ** 120).to(BF16)
    q[:, 1::2] *= 2.0 ** -40
    off, context = ints([0, new]), ints([L])
    got = attention.attend(q, cache, table, off, context, scale=0.25)
    ref.check_attend(got, q, cache, table, off, context, 0.25)
    # a scale that makes every row large, of tiles that rows do not fill
    got = attention.attend((q.double() * 2.0 ** -120).to(BF16), cache, table, off, context,
                           scale=2.0 ** 118)
    ref.check_attend(got, (q.double() * 2.0 ** -120).to(BF16), cache, table, off, context, 2.0 ** 118)
    assert experts.status() == ciera.OK
