"""What the attention half's entry points refuse, checked without a GPU (the
checks come before any CUDA call, and the fake pointers are never followed), and
the frequencies of rotary tables."""
import ctypes
import math

import pytest
import torch

from lossless_exponent_reuse_gb300 import attention, ciera, experts

FAKE, ODD = 4096, 4097


def vp(v):
    return None if v is None else ctypes.c_void_p(v)


def rotary(x=FAKE, xt=256, xh=64, at=FAKE, turns=FAKE, pairs=32, amp=1.0, tokens=3, heads=4, dim=64,
           y=2 * FAKE, yt=256, yh=64, flags=0):
    return ciera.lib().ciera_rotary(vp(x), xt, xh, vp(at), vp(turns), pairs, amp, tokens, heads,
                                    dim, vp(y), yt, yh, flags, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=ODD), dict(at=None), dict(at=4098), dict(turns=None), dict(turns=4100),
    dict(pairs=33), dict(pairs=-1), dict(amp=float("nan")), dict(amp=float("inf")),
    dict(tokens=-1), dict(heads=-1), dict(dim=-1), dict(dim=1025, xh=2000, xt=9000), dict(y=None),
    dict(y=ODD), dict(yh=63), dict(yt=255), dict(yt=64, yh=64), dict(yt=0), dict(flags=4),
    dict(xt=-1), dict(xh=1 << 41), dict(tokens=1 << 29, heads=8),
    dict(y=FAKE, yt=512)])
def test_rotary_refuses(bad):
    assert rotary(**bad) == ciera.E_INVAL


def test_rotary_of_nothing_is_nothing():
    assert rotary(tokens=0, x=None, y=None, at=None) == ciera.OK
    assert rotary(heads=0, x=None, y=None) == ciera.OK
    assert rotary(dim=0, pairs=0, turns=None) == ciera.OK


def cache(key=FAKE, value=FAKE, ke=0, ve=0, ks=(1024, 128, 64), vs=(1024, 128, 64), kes=(0, 0, 0),
          ves=(0, 0, 0), pages=5, page=8, heads=2, dim=64, kind=experts.BF16):
    return attention._cache_words(key, value, ke, ve, *ks, *vs, *kes, *ves, pages, page, heads, dim,
                                  kind)


E4M3 = dict(kind=experts.E4M3, ke=FAKE, ve=FAKE, kes=(16, 2, 1), ves=(16, 2, 1))
BAD_CACHES = [
    dict(key=0), dict(key=ODD), dict(value=0), dict(kind=experts.F32), dict(kind=9), dict(pages=-1),
    dict(page=0), dict(heads=-1), dict(dim=-1), dict(pages=1 << 20, page=1 << 12), dict(ke=FAKE),
    {**E4M3, "ke": 0}, {**E4M3, "ve": 0}, {**E4M3, "kes": (-1, 2, 1)}, dict(ks=(-1, 128, 64)),
    dict(vs=(1 << 41, 128, 64))]


def append(q=FAKE, qt=256, qh=64, k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, at=FAKE, slots=FAKE,
           turns=FAKE, pairs=32, amp=1.0, tokens=3, heads=4, out=2 * FAKE, ot=256, oh=64, flags=0,
           c=None):
    return ciera.lib().ciera_append(vp(q), qt, qh, vp(k), kt, kh, vp(v), vt, vh, vp(at), vp(slots),
                                    vp(turns), pairs, amp, tokens, heads, vp(out), ot, oh,
                                    cache() if c is None else c, flags, None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(q=ODD), dict(k=None), dict(v=None), dict(at=None), dict(slots=None),
    dict(slots=4098), dict(turns=None), dict(pairs=33), dict(amp=float("inf")), dict(tokens=-1),
    dict(heads=-1), dict(out=None), dict(oh=60), dict(flags=2), dict(kt=-1), dict(vh=-1),
    dict(tokens=1 << 28, heads=8), dict(out=FAKE, ot=300)])
def test_append_refuses(bad):
    assert append(**bad) == ciera.E_INVAL


@pytest.mark.parametrize("bad", BAD_CACHES + [
    dict(ks=(1023, 128, 64)), dict(vs=(1024, 127, 64)), dict(ks=(1024, 128, 63)),
    {**E4M3, "kes": (15, 2, 1)}, {**E4M3, "ves": (16, 1, 1)}])
def test_append_refuses_caches(bad):
    assert append(c=cache(**bad)) == ciera.E_INVAL


def test_append_refuses_no_cache_and_takes_none():
    assert ciera.lib().ciera_append(
        vp(FAKE), 256, 64, vp(FAKE), 128, 64, vp(FAKE), 128, 64, vp(FAKE), vp(FAKE), vp(FAKE), 32,
        1.0, 3, 4, vp(2 * FAKE), 256, 64, None, 0, None) == ciera.E_INVAL
    assert append(tokens=0, q=None, k=None, v=None, at=None, slots=None, out=None) == ciera.OK


def pages(cached=FAKE, new=FAKE, requests=3, tokens=10, page=16, table=FAKE, ts=8, width=8,
          free=FAKE, capacity=9, count=FAKE, left=FAKE, off=FAKE, ctx=FAKE, lens=FAKE, pos=FAKE,
          slots=FAKE):
    return ciera.lib().ciera_assign_pages(
        vp(cached), vp(new), requests, tokens, page, vp(table), ts, width, vp(free), capacity,
        vp(count), vp(left), vp(off), vp(ctx), vp(lens), vp(pos), vp(slots), None)


@pytest.mark.parametrize("bad", [
    dict(cached=None), dict(new=4098), dict(requests=-1), dict(requests=(1 << 20) + 1),
    dict(tokens=-1), dict(page=0), dict(table=None), dict(ts=7), dict(width=-1), dict(free=None),
    dict(capacity=-1), dict(count=None), dict(left=None), dict(off=None), dict(ctx=None),
    dict(lens=None), dict(pos=None), dict(slots=None), dict(slots=4097)])
def test_assign_pages_refuses(bad):
    assert pages(**bad) == ciera.E_INVAL


@pytest.mark.parametrize("bad", [
    dict(done=None), dict(lens=None), dict(requests=-1), dict(page=0), dict(table=None), dict(ts=7),
    dict(free=None), dict(capacity=-1), dict(count=None), dict(left=4098)])
def test_release_pages_refuses(bad):
    a = dict(done=FAKE, lens=FAKE, requests=3, page=16, table=FAKE, ts=8, width=8, free=FAKE,
             capacity=9, count=FAKE, left=FAKE)
    a.update(bad)
    assert ciera.lib().ciera_release_pages(
        vp(a["done"]), vp(a["lens"]), a["requests"], a["page"], vp(a["table"]), a["ts"], a["width"],
        vp(a["free"]), a["capacity"], vp(a["count"]), vp(a["left"]), None) == ciera.E_INVAL


def attend(q=FAKE, qt=256, qh=64, tokens=3, heads=4, c=None, table=FAKE, ts=8, width=8, off=FAKE,
           ctx=FAKE, requests=2, longest=3, scale=0.125, o=FAKE, ws=FAKE, size=None, ctl=FAKE):
    L = ciera.lib()
    size = L.ciera_attend_workspace_bytes(4, 2, 64) if size is None else size
    return L.ciera_attend(vp(q), qt, qh, tokens, heads, cache() if c is None else c, vp(table), ts,
                          width, vp(off), vp(ctx), requests, longest, scale, vp(o), vp(ws), size,
                          vp(ctl), None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(q=ODD), dict(qt=-1), dict(tokens=-1), dict(heads=3), dict(heads=1),
    dict(heads=0), dict(table=None), dict(table=4098), dict(ts=7), dict(width=-1), dict(off=None),
    dict(ctx=None), dict(requests=-1), dict(longest=-1), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(o=None), dict(o=ODD), dict(ws=None), dict(ws=4100), dict(size=100),
    dict(ctl=None), dict(ctl=4098), dict(tokens=1 << 30)])
def test_attend_refuses(bad):
    assert attend(**bad) == ciera.E_INVAL


@pytest.mark.parametrize("bad", BAD_CACHES + [dict(heads=0), dict(dim=0), dict(dim=257)])
def test_attend_refuses_caches(bad):
    assert attend(c=cache(**bad)) == ciera.E_INVAL


def test_attend_of_nothing_is_nothing():
    assert attend(tokens=0, q=None, o=None) == ciera.OK


def test_attend_workspace():
    need = ciera.lib().ciera_attend_workspace_bytes
    assert need(16, 16, 128) >= need(16, 16, 256) > 0
    for bad in ((0, 0, 64), (4, 3, 64), (2, 4, 64), (-4, 2, 64), (4, 2, 0), (4, 2, 257), (4, -2, 64)):
        assert need(*bad) == 0


# ---- the binding's own checks, on tensors that are not on a GPU ---------------

def test_binding_refuses_what_is_not_on_a_gpu():
    x, at = torch.zeros(2, 3, 8, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    r = attention.rotary_table(8, device="cpu")
    c = attention.page_cache(2, 4, 1, 8, device="cpu")
    pool = attention.page_pool(4, 2, 2, device="cpu")
    for call in (lambda: attention.rotary(x, at, r), lambda: attention.rotary_backward(x, at, r),
                 lambda: attention.append(x, x, x, at, at, r, c),
                 lambda: attention.attend(x, c, pool.table, at, at),
                 lambda: attention.assign_pages(pool, at, at, 2, 4),
                 lambda: attention.release_pages(pool, at, at.bool(), 4)):
        with pytest.raises(ValueError):
            call()


def test_cache_layout_matches_the_header():
    from test_lib_host import _c_layout
    fields = ["key_dev", "value_dev", "key_exponent_dev", "value_exponent_dev", "key_stride",
              "value_stride", "key_exponent_stride", "value_exponent_stride", "pages", "page_size",
              "heads", "head_dim", "type"]
    size, offsets = _c_layout("ciera_cache", fields)
    words = [0, 1, 2, 3, 4, 7, 10, 13, 16, 17, 18, 19, 20]
    assert size == len(cache()) == 168 and offsets == [8 * w for w in words]


def test_caches_and_pools_as_made():
    c = attention.page_cache(3, 4, 2, 16, device="cpu")
    assert c.key.shape == (3, 4, 2, 16) and c.key.stride() == (128, 16, 64, 1)
    assert c.key_exponent is None and c.key.data_ptr() != c.value.data_ptr()
    c = attention.page_cache(3, 4, 2, 16, e4m3=True, device="cpu")
    assert c.key.dtype == torch.float8_e4m3fn and c.value_exponent.shape == (3, 4, 2)
    pool = attention.page_pool(5, 2, 3, device="cpu")
    assert pool.free.tolist() == [4, 3, 2, 1, 0] and int(pool.count) == 5
    assert (pool.table == -1).all() and pool.table.shape == (2, 3)


# ---- frequencies ---------------------------------------------------------------

def radians(r):
    return [(t % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for t in r.turns.tolist()]


def test_frequencies():
    r = attention.rotary_table(16, device="cpu")
    assert radians(r) == pytest.approx([10000 ** (-i / 8) for i in range(8)], rel=1e-15)
    assert r.amplitude == 1.0 and not r.interleaved
    given = attention.rotary_table(6, frequencies=[0.5, -0.25, 7.0], device="cpu", interleaved=True,
                                   amplitude=2.0)
    assert radians(given) == pytest.approx([0.5, 2 * math.pi - 0.25, 7.0 - 2 * math.pi], rel=1e-14)
    assert given.amplitude == 2.0 and given.interleaved
    assert attention.rotary_table(0, device="cpu").turns.numel() == 0


def test_scaled_frequencies():
    plain = radians(attention.rotary_table(64, device="cpu"))
    linear = radians(attention.rotary_table(64, scaling="linear", factor=4, device="cpu"))
    assert linear == pytest.approx([w / 4 for w in plain], rel=1e-14)
    base = radians(attention.rotary_table(64, scaling="base", factor=4, device="cpu"))
    assert base[0] == pytest.approx(plain[0]) and base[-1] == pytest.approx(plain[-1] / 4, rel=1e-12)
    parts = attention.rotary_table(64, scaling="parts", factor=4, original=2048, device="cpu")
    for w, got in zip(plain, radians(parts)):
        turns = 2048 * w / (2 * math.pi)
        keep = min(1, max(0, (turns - 1) / 31))
        assert got == pytest.approx(w * keep + w / 4 * (1 - keep), rel=1e-13)
    assert parts.amplitude == pytest.approx(1 + 0.1 * math.log(4))
    assert attention.rotary_table(2, scaling="base", factor=9, device="cpu").turns.numel() == 1


@pytest.mark.parametrize("bad", [
    dict(dim=7), dict(dim=-2), dict(base=0), dict(base=math.inf), dict(scaling="some"),
    dict(scaling="parts", factor=2), dict(scaling="parts", factor=2, original=9, bounds=(3, 3)),
    dict(factor=0.5), dict(factor=math.inf), dict(frequencies=[1.0]),
    dict(frequencies=[math.nan] * 4), dict(scaling="base", frequencies=[1.0] * 4)])
def test_rotary_table_refuses(bad):
    with pytest.raises(ValueError):
        attention.rotary_table(**{"dim": 8, "device": "cpu", **bad})


@pytest.mark.parametrize("head_dim,rows,o", [(96, (256, 128), None), (0, (256, 128), None),
                                             (64, (256, 100), None), (64, (256, 128), (256, 64))])
def test_layer_refuses_heads_that_its_weights_do_not_have(head_dim, rows, o):
    import dataclasses

    from lossless_exponent_reuse_gb300 import moe_layer, workloads
    wl = moe_layer.layer_workload(2, 64, 32, ranks=1, block=64, attention_rows=rows)
    if o:
        wl = dataclasses.replace(wl, tensors=tuple(
            workloads.Tensor(t.name, o) if t.name == "attn.o" else t for t in wl.tensors))
    bucket, turn = torch.zeros(wl.numel, dtype=torch.bfloat16), attention.rotary_table(8, device="cpu")
    with pytest.raises(ValueError):
        moe_layer.AttentionLayer(bucket, wl, head_dim, turn)
