"""Attention over pages against the definition in 64 bits, on every form that a
call can take."""
import math

import pytest
import torch

import attention_reference as ref
from attention_reference import BF16, ints, rand
from lossless_exponent_reuse_gb300 import attention, ciera, experts

pytestmark = pytest.mark.gpu


def batch(new, cached, q_heads, heads, dim, page, seed=1, **how):
    lengths = [n + c for n, c in zip(new, cached)]
    cache, table = ref.paged(lengths, page, heads, dim, seed=seed, **how)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    q = rand(offsets[-1], q_heads, dim, seed=seed + 77, scale=2.0)
    return q, cache, table, ints(offsets), ints(lengths)


def run(new, cached, q_heads, heads, dim, page, **how):
    q, cache, table, offsets, context = batch(new, cached, q_heads, heads, dim, page, **how)
    got = attention.attend(q, cache, table, offsets, context, longest=max(new))
    ref.check_attend(got, q, cache, table, offsets, context,
                     what=(new, cached, q_heads, heads, dim, page, how))
    assert experts.status() == ciera.OK


HEADS = [(16, 16), (8, 1), (12, 4), (3, 3)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim", [64, 80, 96, 128, 256])
@pytest.mark.parametrize("q_heads,heads", HEADS)
def test_single_tokens(q_heads, heads, dim, e4m3):
    run([1] * 5, [0, 1, 15, 16, 300], q_heads, heads, dim, 16, e4m3=e4m3)
    run([1] * 3, [1000, 63, 2049], q_heads, heads, dim, 64, e4m3=e4m3, by_head=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 20, 24, 40, 64, 128, 136, 192, 256])
def test_page_sizes(page, e4m3):
    run([1, 5, 33], [127, 128, 300], 8, 4, 128, page, e4m3=e4m3)
    run([130, 1, 270], [0, 500, 129], 4, 2, 64, page, e4m3=e4m3, by_head=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [1, 2, 3, 4, 5, 6, 7, 10, 17, 20, 34, 50, 63, 65, 100, 127, 129,
                                  131, 250])
def test_many_rows_of_odd_pages(page, e4m3):
    """Pages whose parts begin at any row of a stage, or that none of a size divide."""
    run([150, 1, 290], [77, 200, 0], 4, 2, 128, page, e4m3=e4m3)
    run([40, 129], [300, 1], 6, 1, 64, page, e4m3=e4m3, by_head=True)
    run([60], [400], 2, 1, 80, page, e4m3=e4m3)
    # keys and values behind the last one
    q, cache, table, offsets, context = batch([140], [71], 4, 2, 128, page)
    L = 211
    at = table[0, (L - 1) // page].long()
    cache.value[at, (L - 1) % page + 1:] = math.nan
    cache.key[at, (L - 1) % page + 1:] = math.inf
    cache.value[at, (L - 1) % page, 1, 3] = math.inf      # the last token alone sees it
    got = attention.attend(q, cache, table, offsets, context)
    ref.check_attend(got, q, cache, table, offsets, context)
    assert torch.isfinite(got[:139]).all()


@pytest.mark.parametrize("dim", [64, 72, 80, 96, 112, 128, 256])
@pytest.mark.parametrize("q_heads,heads", HEADS)
def test_chunks(q_heads, heads, dim):
    e4m3 = dim % 16 == 0 and q_heads == 12
    run([17, 64, 1, 0, 130], [0, 5, 700, 9, 127], q_heads, heads, dim, 16, e4m3=e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new", [127, 128, 129, 255, 256, 257, 513])
def test_prompts(new, e4m3):
    run([new], [0], 4, 4, 128, 16, e4m3=e4m3)
    run([new, new + 1], [new, 3], 6, 2, 64, 32, e4m3=e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", range(1, 36, 2))
def test_rows_per_head_around_every_tile(rows, e4m3):
    run([rows, 1], [200, 77], 2, 2, 128, 16, e4m3=e4m3)
    run([rows], [1], 5, 1, 96, 16, e4m3=e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
def test_long_contexts_over_all_blocks(e4m3):
    run([1], [20000], 16, 2, 128, 16, e4m3=e4m3)
    run([64], [9000], 8, 1, 128, 64, e4m3=e4m3)
    run([1, 200, 1], [5, 4000, 7000], 8, 8, 64, 32, e4m3=e4m3)


def test_many_requests():
    g = torch.Generator().manual_seed(5)
    cached = torch.randint(0, 200, (700,), generator=g).tolist()
    run([1] * 700, cached, 4, 2, 64, 16)
    new = torch.randint(0, 40, (300,), generator=g).tolist()
    run(new, cached[:300], 4, 1, 64, 16)


def test_an_order_of_requests_changes_no_row():
    """A batch's rows are those that each request has alone."""
    new, cached = [3, 200, 1, 40, 1, 1], [500, 0, 3000, 77, 15, 16]
    q, cache, table, off, context = batch(new, cached, 8, 2, 128, 16)
    got = attention.attend(q, cache, table, off, context)
    for r, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        one = attention.attend(q[a:b], cache, table[r:r + 1], ints([0, b - a]), context[r:r + 1])
        assert (got[a:b].float() - one.float()).norm() <= 2.0 ** -7 * one.float().norm()


def test_nothing():
    q, cache, table, offsets, context = batch([3, 2], [0, 1], 4, 2, 64, 16)
    none = attention.attend(q[:0], cache, table, ints([0, 0, 0]), context)
    assert none.shape == (0, 4, 64)
    got = attention.attend(q, cache, table[:0], ints([0]), context[:0])
    assert (got == 0).all()
    got = attention.attend(q, cache, table, offsets, ints([0, 0]))
    assert (got == 0).all()
    got = attention.attend(q, cache, table[:, :0], offsets, context)
    assert (got == 0).all()
    assert experts.status() == ciera.OK


@pytest.mark.parametrize("dim,page", [(128, 16), (64, 20), (66, 16)])
def test_rows_that_see_nothing_and_rows_behind_the_last(dim, page):
    # more new tokens than keys: the first see none
    q, cache, table, _, _ = batch([300, 40, 9], [0, 0, 20], 4, 2, dim, page)
    offsets, context = ints([0, 250, 290, 299]), ints([100, 0, 29])
    got = attention.attend(q, cache, table, offsets, context)
    ref.check_attend(got, q, cache, table, offsets, context)
    assert (got[:150] == 0).all() and (got[250:290] == 0).all() and (got[299:] == 0).all()
    assert (got[150:250].float().abs().amax((1, 2)) > 0).all()


@pytest.mark.parametrize("longest", [None, 1, 40, 10 ** 9])
def test_longest_changes_no_row(longest):
    q, cache, table, offsets, context = batch([40, 1, 7], [100, 300, 0], 8, 2, 128, 16)
    got = attention.attend(q, cache, table, offsets, context, longest=longest)
    ref.check_attend(got, q, cache, table, offsets, context, what=longest)


@pytest.mark.parametrize("new,page,dim,e4m3", [
    (1, 16, 128, False), (1, 20, 64, True), (150, 16, 128, False), (150, 24, 80, True),
    (150, 20, 128, False), (300, 128, 64, False)])
def test_each_row_finds_its_key(new, page, dim, e4m3):
    """Row i's query has one key that outweighs all others, and one almost as great
    just out of its sight."""
    cached, heads = 437, 2
    L = cached + new
    g = torch.Generator(device="cuda").manual_seed(3)
    key = torch.randn(L, heads, dim, generator=g, device="cuda").sign() * 0.5
    rows = {0: key, 1: torch.randn(L, heads, dim, generator=g, device="cuda")}
    cache, table = ref.paged([L], page, heads, dim, e4m3=e4m3,
                             value=lambda kind, r, n: rows[kind])
    at = torch.arange(L, device="cuda")
    slot = table[0].long()[at // page], at % page
    if e4m3:
        K = ref.values(cache.key.view(torch.uint8)[slot].view(cache.key.dtype),
                       cache.key_exponent[slot])
        K = K / K.norm(dim=2, keepdim=True) * 4
    else:
        K = ref.values(cache.key[slot], None)
    i = torch.arange(new, device="cuda")
    for target in (cached + i, i * 0, cached + i - 1, (i * 37 + 5) % (cached + 1), 0 * i + cached - 1):
        for scale in (1.0, 20.0):
            hidden = torch.clamp(cached + i + 1, max=L - 1)
            q = (K[target] * scale + K[hidden] * scale * 0.9).to(BF16)
            got = attention.attend(q, cache, table, ints([0, new]), ints([L]), scale=1.0)
            ref.check_attend(got, q, cache, table, ints([0, new]), ints([L]), scale=1.0)


@pytest.mark.parametrize("new,page,dim,q_heads", [
    (5, 16, 128, 4), (140, 16, 128, 2), (140, 24, 64, 4), (37, 20, 128, 2), (12, 16, 66, 2)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_out_of_sight_have_no_part(new, page, dim, q_heads, bad):
    q, cache, table, offsets, context = batch([new, 3], [70, 11], q_heads, 2, dim, page)
    L = 70 + new
    for key, d in ((L - 1, 3), (L - 2, 0), (70, dim - 1)):
        cache.value[table[0, key // page].long(), key % page, 1, d] = bad
    cache.key[table[0, (L - 1) // page].long(), (L - 1) % page, 1, 2] = math.nan
    got = attention.attend(q, cache, table, offsets, context)
    ref.check_attend(got, q, cache, table, offsets, context)
    # the other head, the other request
    assert torch.isfinite(got[:, :q_heads // 2]).all() and torch.isfinite(got[new:]).all()


@pytest.mark.parametrize("q_heads,new,page,dim,longest", [
    (48, 2, 20, 128, None), (40, 3, 20, 64, None), (24, 2, 16, 256, None), (12, 2, 16, 128, 1),
    (9, 3, 20, 64, 1), (48, 2, 1, 128, None), (40, 3, 1, 64, None)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_tiles_that_begin_and_end_inside_a_token(q_heads, new, page, dim, longest, bad):
    """Of fewer rows than a token has, but of two tokens, the first of which does
    not see the second's key."""
    q, cache, table, offsets, context = batch([new], [50], q_heads, 1, dim, page)
    L = 50 + new
    cache.value[table[0, (L - 1) // page].long(), (L - 1) % page, 0, 3] = bad
    got = attention.attend(q, cache, table, offsets, context, longest=longest)
    ref.check_attend(got, q, cache, table, offsets, context)
    assert torch.isfinite(got[:new - 1]).all()


@pytest.mark.parametrize("new,page,dim", [(1, 16, 128), (3, 20, 64), (200, 16, 128), (200, 24, 64)])
def test_rows_of_any_exponent(new, page, dim):
    """Powers of two from the lowest to the highest, zeros, and NaN by exponent and by
    value, on keys and on values."""
    L, heads = new + 260, 2
    cache, table = ref.paged([L], page, heads, dim, e4m3=True)
    at = torch.arange(L, device="cuda")
    slot = table[0].long()[at // page], at % page
    e = torch.randint(27, 135, (L, heads), generator=torch.Generator().manual_seed(1)).cuda()
    e[::5] = torch.randint(120, 130, (len(e[::5]), heads)).cuda()
    e[7], e[11] = 0, 245                     # of which only the values are small
    small = cache.value.view(torch.uint8)
    small[slot[0][11], slot[1][11]] = 0
    cache.value_exponent[slot] = e.to(torch.uint8)
    k = torch.full((L, heads), 121, dtype=torch.uint8, device="cuda")
    k[::9], k[3] = 27, 0
    cache.key_exponent[slot] = k
    q = rand(new, 4, dim, seed=4)
    off, context = ints([0, new]), ints([L])
    got = attention.attend(q, cache, table, off, context)
    ref.check_attend(got, q, cache, table, off, context)
    cache.value_exponent[slot[0][L - 1], slot[1][L - 1], 0] = 255      # the last row alone sees it
    small[slot[0][L - 1], slot[1][L - 1], 1, 5] = 0xFF
    got = attention.attend(q, cache, table, off, context)
    ref.check_attend(got, q, cache, table, off, context)
    assert torch.isnan(got[-1, :2]).all() and torch.isnan(got[-1, 2:, 5]).all()
    assert torch.isfinite(got[:-1]).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_scores_that_rise_and_fall(e4m3):
    """Maxima that grow from tile to tile, by much and by little, and fall."""
    L, heads, dim = 3000, 2, 128
    for slope in (0.01, 0.3, -0.3):
        ramp = torch.arange(L, device="cuda", dtype=torch.float32) * slope
        rows = lambda kind, r, n: (ramp[:, None, None].expand(L, heads, dim) / 256 + rand(
            L, heads, dim, seed=9 + kind, dtype=torch.float32, scale=0.1))
        cache, table = ref.paged([L], 16, heads, dim, e4m3=e4m3, value=rows)
        for new in (1, 200):
            q = torch.ones(new, heads, dim, device="cuda", dtype=BF16)
            got = attention.attend(q, cache, table, ints([0, new]), ints([L]), scale=0.5)
            ref.check_attend(got, q, cache, table, ints([0, new]), ints([L]), scale=0.5)


def test_pages_that_are_not_there_hold_zeros():
    q, cache, table, offsets, context = batch([1, 40, 200], [300, 100, 90], 4, 2, 128, 16)
    table[0, 3], table[1, 0], table[2, 2] = -1, cache.key.shape[0], 2 ** 31 - 1
    table[2, 0] = -2 ** 31
    got = attention.attend(q, cache, table, offsets, context)
    ref.check_attend(got, q, cache, table, offsets, context)


def test_lengths_and_offsets_out_of_range():
    q, cache, table, _, _ = batch([50, 30, 1], [10, 60, 90], 4, 2, 64, 16)
    cache.key.nan_to_num_(0), cache.value.nan_to_num_(0)
    for offsets, context in (([7, 50, 80, 81], [60, 90, 10 ** 9]),
                             ([0, 50, 10 ** 9, 10 ** 9], [60, 90, 91]),
                             ([0, -5, 80, 81], [60, -3, 91])):
        got = attention.attend(q, cache, table, ints(offsets), ints(context))
        ref.check_attend(got, q, cache, table, ints(offsets), ints(context))


@pytest.mark.parametrize("how", ["q view", "odd q", "table view", "cache view", "odd cache",
                                 "values elsewhere"])
@pytest.mark.parametrize("new", [1, 150])
def test_layouts(how, new):
    q, cache, table, offsets, context = batch([new, 4], [200, 31], 4, 2, 128, 16)
    T = q.shape[0]
    if how == "q view":
        wide = torch.full((T, 9, 128), math.nan, device="cuda", dtype=BF16)
        wide[:, 2:6] = q
        q = wide[:, 2:6]
    if how == "odd q":
        wide = torch.full((T, 4, 131), math.nan, device="cuda", dtype=BF16)
        wide[:, :, 1:129] = q
        q = wide[:, :, 1:129]
    if how == "table view":
        wide = torch.full((2, table.shape[1] + 5), 10 ** 9, device="cuda", dtype=torch.int32)
        wide[:, :table.shape[1]] = table
        table = wide[:, :table.shape[1]]
    if how in ("cache view", "odd cache"):
        pad = 8 if how == "cache view" else 3
        shape = cache.key.shape
        wide = torch.full((shape[0], 16, 5, 128 + pad), math.nan, device="cuda", dtype=BF16)
        wide[:, :, 1:3, :128], wide[:, :, 3:5, :128] = cache.key, cache.value
        cache = attention.Cache(wide[:, :, 1:3, :128], wide[:, :, 3:5, :128])
    if how == "values elsewhere":
        cache = attention.Cache(cache.key, cache.value.transpose(1, 2).contiguous().transpose(1, 2))
    got = attention.attend(q, cache, table, offsets, context)
    ref.check_attend(got, q, cache, table, offsets, context, what=how)


def test_heads_of_any_size():
    for dim in (1, 7, 8, 16, 24, 33, 130, 200, 250):
        run([3, 20], [10, 40], 4, 2, dim, 16)
    for dim in (16, 24, 48, 240):
        run([3, 20], [10, 40], 4, 2, dim, 16, e4m3=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_heads,heads", [(128, 1), (200, 1), (256, 1), (130, 2), (64, 2)])
def test_many_query_heads_to_one(q_heads, heads, e4m3):
    run([1, 5, 2], [300, 40, 0], q_heads, heads, 128, 16, e4m3=e4m3)
    run([1], [700], q_heads, heads, 64, 24, e4m3=e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-30, 3.0])
def test_scales(scale, e4m3):
    for new in (1, 150):
        q, cache, table, off, context = batch([new, 3], [200, 31], 4, 2, 128, 16, e4m3=e4m3)
        got = attention.attend(q, cache, table, off, context, scale=scale)
        ref.check_attend(got, q, cache, table, off, context, scale=scale)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_cache_of_no_pages_holds_zeros(e4m3):
    cache = attention.page_cache(0, 16, 2, 128, e4m3=e4m3)
    for new in (1, 200):
        q, table = rand(new, 4, 128), torch.zeros(1, 20, dtype=torch.int32, device="cuda")
        got = attention.attend(q, cache, table, ints([0, new]), ints([new + 5]))
        assert (got == 0).all()
    assert experts.status() == ciera.OK


def test_rows_of_nan_are_nan_alone():
    """Queries and keys of NaN, in rows that everyone computes together."""
    for new in (9, 300):
        q, cache, table, off, context = batch([new, 40], [100, 60], 4, 2, 128, 16)
        q[3, 1] = math.nan
        q[new + 2, 0, 5] = math.inf
        cache.key[table[1, 1].long(), 3, 1, 7] = math.nan       # all of request 1's head 1 see it
        got = attention.attend(q, cache, table, off, context)
        odd = torch.isnan(got).all(2)
        want = torch.zeros_like(odd)
        want[3, 1] = want[new + 2, 0] = True
        want[new:, 2:] = True
        assert torch.equal(odd, want) and torch.isfinite(got[~want]).all()
        q[3, 1], q[new + 2, 0, 5] = 1.0, 1.0
        cache.key[table[1, 1].long(), 3, 1, 7] = 1.0
        clean = attention.attend(q, cache, table, off, context)
        assert torch.equal(got[~want], clean[~want])


def test_places_behind_32_bits():
    """A cache of more than 2^32 values, of which a few pages are used."""
    pages, page, heads, dim = 2200, 512, 32, 128
    cache = attention.Cache(*(torch.empty(pages, page, heads, dim, dtype=BF16, device="cuda")
                              for _ in range(2)))
    L, picked = 1300, [pages - 1, 3, pages - 2]
    at = torch.tensor(picked, device="cuda")
    for side, seed in ((cache.key, 1), (cache.value, 2)):
        side[at] = rand(3 * page, heads, dim, seed=seed).view(3, page, heads, dim)
    small = attention.Cache(*(s[at] for s in cache[:2]))
    for new in (1, 130):
        q = rand(new, heads, dim, seed=3, scale=2.0)
        got = attention.attend(q, cache, ints([picked]), ints([0, new]), ints([L]))
        ref.check_attend(got, q, small, ints([[0, 1, 2]]), ints([0, new]), ints([L]))


def test_same_results_every_time():
    q, cache, table, offsets, context = batch([1, 300, 20, 1], [9000, 100, 3000, 50], 8, 2, 128, 16)
    first = attention.attend(q, cache, table, offsets, context)
    for _ in range(5):
        assert torch.equal(first, attention.attend(q, cache, table, offsets, context))
