"""What the mixture-of-experts entry points refuse, checked without a GPU: the
checks come before any CUDA call, and the fake pointers are never followed."""
import ctypes

import pytest
import torch

from lossless_exponent_reuse_gb300 import ciera, experts, workloads

FAKE, ODD = 4096, 4097


def vp(v):
    return None if v is None else ctypes.c_void_p(v)


def norm(L, x=FAKE, xs=64, res=None, rs=0, w=FAKE, rows=4, dim=64, eps=1e-6, y=FAKE,
         kind=experts.BF16, scale=None, h=None, rstd=None):
    return L.ciera_rmsnorm(vp(x), xs, vp(res), rs, vp(w), rows, dim, eps, vp(y), kind, vp(scale),
                           vp(h), vp(rstd), None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=ODD), dict(xs=63), dict(w=None), dict(rows=-1), dict(dim=-1),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(y=None),
    dict(kind=experts.F32), dict(kind=9), dict(kind=experts.E4M3), dict(scale=FAKE),
    dict(res=FAKE, rs=8), dict(res=ODD, rs=64), dict(res=FAKE, rs=72, h=FAKE), dict(h=ODD),
    dict(rstd=4098), dict(dim=1 << 40, xs=1 << 41)])
def test_norm_refuses(bad):
    assert norm(ciera.lib(), **bad) == ciera.E_INVAL


def test_norm_of_nothing_is_nothing():
    assert norm(ciera.lib(), rows=0, x=None, y=None) == ciera.OK
    assert ciera.lib().ciera_quantize_rows(None, 8, 0, 8, None, None, None) == ciera.OK


@pytest.mark.parametrize("bad", [dict(x=None), dict(x=ODD), dict(xs=7), dict(y=None),
                                 dict(scale=None), dict(scale=4098)])
def test_quantize_rows_refuses(bad):
    a = dict(x=FAKE, xs=8, y=FAKE, scale=FAKE)
    a.update(bad)
    assert ciera.lib().ciera_quantize_rows(vp(a["x"]), a["xs"], 3, 8, vp(a["y"]), vp(a["scale"]),
                                           None) == ciera.E_INVAL


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(ds=8), dict(h=None), dict(hs=8), dict(rstd=None), dict(w=None),
    dict(dh=FAKE, dhs=3), dict(dx=None), dict(dw=None), dict(ws=None), dict(ws=4100),
    dict(size=0), dict(rows=-2), dict(rows=1 << 33)])
def test_norm_gradient_refuses(bad):
    L = ciera.lib()
    a = dict(dy=FAKE, ds=64, h=FAKE, hs=64, rstd=FAKE, w=FAKE, dh=None, dhs=0, rows=10, dim=64,
             dx=FAKE, dw=FAKE, ws=FAKE, size=L.ciera_moe_workspace_bytes(10, 0, 64))
    a.update(bad)
    assert L.ciera_rmsnorm_backward(
        vp(a["dy"]), a["ds"], vp(a["h"]), a["hs"], vp(a["rstd"]), vp(a["w"]), vp(a["dh"]),
        a["dhs"], a["rows"], a["dim"], vp(a["dx"]), vp(a["dw"]), vp(a["ws"]), a["size"],
        None) == ciera.E_INVAL


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(kind=experts.E4M3), dict(ls=63), dict(tokens=-1), dict(E=0),
    dict(E=1025, ls=2000), dict(k=0), dict(k=33), dict(E=4, k=5), dict(flags=2),
    dict(tokens=1 << 30, k=8), dict(weights=None), dict(chosen=None), dict(slots=None),
    dict(row_tokens=None), dict(offsets=None), dict(ws=None), dict(size=100),
    dict(logits=4098)])
def test_route_refuses(bad):
    L = ciera.lib()
    a = dict(logits=FAKE, kind=experts.F32, ls=64, tokens=10, E=64, k=8, flags=0, weights=FAKE,
             chosen=FAKE, slots=FAKE, row_tokens=FAKE, offsets=FAKE, ws=FAKE,
             size=L.ciera_moe_workspace_bytes(10, 64, 0))
    a.update(bad)
    assert L.ciera_route(vp(a["logits"]), a["kind"], a["ls"], None, a["tokens"], a["E"], a["k"],
                         a["flags"], vp(a["weights"]), vp(a["chosen"]), vp(a["slots"]),
                         vp(a["row_tokens"]), vp(a["offsets"]), vp(a["ws"]), a["size"],
                         None) == ciera.E_INVAL


@pytest.mark.parametrize("bad", [dict(dweights=None), dict(weights=None), dict(chosen=None),
                                 dict(logits=None), dict(kind=7), dict(k=40), dict(flags=4),
                                 dict(dlogits=None), dict(ls=3)])
def test_route_gradient_refuses(bad):
    a = dict(dweights=FAKE, weights=FAKE, chosen=FAKE, logits=FAKE, kind=experts.BF16, ls=64,
             k=8, flags=0, dlogits=FAKE)
    a.update(bad)
    assert ciera.lib().ciera_route_backward(
        vp(a["dweights"]), vp(a["weights"]), vp(a["chosen"]), vp(a["logits"]), a["kind"], a["ls"],
        10, 64, a["k"], a["flags"], vp(a["dlogits"]), None) == ciera.E_INVAL


@pytest.mark.parametrize("bad", [dict(rows=None), dict(rs=7), dict(slots=None), dict(w=4098),
                                 dict(tokens=-1), dict(k=0), dict(k=33), dict(y=None),
                                 dict(dy=None), dict(ds=7), dict(offsets=None), dict(E=2000),
                                 dict(drows=None), dict(dw=None)])
def test_combine_refuses(bad):
    L = ciera.lib()
    a = dict(rows=FAKE, rs=64, n=80, slots=FAKE, w=FAKE, tokens=10, k=8, dim=64, y=FAKE, dy=FAKE,
             ds=64, offsets=FAKE, E=16, drows=FAKE, dw=FAKE)
    a.update(bad)
    if not set(bad) & {"dy", "ds", "offsets", "E", "drows", "dw"}:
        assert L.ciera_combine(vp(a["rows"]), a["rs"], a["n"], vp(a["slots"]), vp(a["w"]),
                               a["tokens"], a["k"], a["dim"], vp(a["y"]), None) == ciera.E_INVAL
    if "y" not in bad:
        assert L.ciera_combine_backward(
            vp(a["dy"]), a["ds"], vp(a["rows"]), a["rs"], a["n"], vp(a["slots"]), vp(a["w"]),
            vp(a["offsets"]), a["E"], a["tokens"], a["k"], a["dim"], vp(a["drows"]),
            vp(a["dw"]), None) == ciera.E_INVAL


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(xs=3), dict(x_rows=99), dict(w=None), dict(ws=3), dict(xscale=FAKE),
    dict(wscale=FAKE), dict(offsets=None), dict(offsets=4098), dict(rows=-1), dict(rows=1 << 31),
    dict(E=1025), dict(E=-1), dict(n=-1), dict(k=-1), dict(kind=experts.F32),
    dict(kind=experts.E4M3), dict(kind=experts.E4M3, xscale=FAKE), dict(flags=2), dict(y=None),
    dict(pre=FAKE), dict(work=None), dict(work=4104), dict(tokens=4098), dict(x=ODD),
    dict(es=-5)])
def test_expert_mm_refuses(bad):
    a = dict(x=FAKE, xs=64, x_rows=100, tokens=None, w=FAKE, ws=64, es=64 * 32, xscale=None,
             wscale=None, offsets=FAKE, rows=100, E=4, n=32, k=64, kind=experts.BF16, flags=0,
             y=FAKE, pre=None, work=FAKE)
    a.update(bad)
    assert ciera.lib().ciera_expert_mm(
        vp(a["x"]), a["xs"], a["x_rows"], vp(a["tokens"]), vp(a["w"]), a["ws"], a["es"],
        vp(a["xscale"]), vp(a["wscale"]), vp(a["offsets"]), a["rows"], a["E"], a["n"], a["k"],
        a["kind"], a["flags"], vp(a["y"]), vp(a["pre"]), vp(a["work"]), None) == ciera.E_INVAL


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(ds=3), dict(w=None), dict(ws=3), dict(offsets=None), dict(rows=-1),
    dict(E=2000), dict(pre=ODD), dict(dx=None), dict(work=None)])
def test_expert_mm_dx_refuses(bad):
    a = dict(dy=FAKE, ds=32, w=FAKE, ws=64, es=64 * 32, offsets=FAKE, rows=100, E=4, n=32, k=64,
             pre=None, dx=FAKE, work=FAKE)
    a.update(bad)
    assert ciera.lib().ciera_expert_mm_dx(
        vp(a["dy"]), a["ds"], vp(a["w"]), a["ws"], a["es"], vp(a["offsets"]), a["rows"], a["E"],
        a["n"], a["k"], vp(a["pre"]), vp(a["dx"]), vp(a["work"]), None) == ciera.E_INVAL


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(ds=3), dict(x=None), dict(xs=3), dict(offsets=None),
    dict(E=2000), dict(dw=None), dict(dws=3), dict(es=3), dict(kind=experts.E4M3),
    dict(kind=experts.F32, dw=4098), dict(flags=1), dict(work=None)])
def test_expert_mm_dw_refuses(bad):
    a = dict(dy=FAKE, ds=32, x=FAKE, xs=64, offsets=FAKE, rows=100, E=4, n=32, k=64, dw=FAKE,
             dws=64, es=64 * 32, kind=experts.BF16, flags=0, work=FAKE)
    a.update(bad)
    assert ciera.lib().ciera_expert_mm_dw(
        vp(a["dy"]), a["ds"], vp(a["x"]), a["xs"], vp(a["offsets"]), a["rows"], a["E"], a["n"],
        a["k"], vp(a["dw"]), a["dws"], a["es"],
        a["kind"], a["flags"], vp(a["work"]), None) == ciera.E_INVAL


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=ODD), dict(xs=7), dict(kind=experts.F32), dict(scale=FAKE),
    dict(yscale=FAKE), dict(kind=experts.E4M3), dict(kind=experts.E4M3, scale=FAKE),
    dict(tokens=None), dict(tokens=4098), dict(rows=-1), dict(y=None), dict(y=ODD)])
def test_gather_rows_refuses(bad):
    a = dict(x=FAKE, xs=8, kind=experts.BF16, scale=None, tokens=FAKE, rows=4, y=FAKE,
             yscale=None)
    a.update(bad)
    assert ciera.lib().ciera_gather_rows(vp(a["x"]), a["xs"], 3, a["kind"], vp(a["scale"]),
                                         vp(a["tokens"]), a["rows"], 8, vp(a["y"]),
                                         vp(a["yscale"]), None) == ciera.E_INVAL


def test_calls_without_rows_need_no_device():
    L = ciera.lib()
    assert L.ciera_expert_mm(None, 8, 0, None, vp(FAKE), 8, 64, None, None, vp(FAKE), 0, 2, 4, 8,
                             experts.BF16, 0, None, None, vp(FAKE), None) == ciera.OK
    assert L.ciera_combine(None, 8, 0, None, None, 0, 1, 8, None, None) == ciera.OK


def test_workspace_bytes():
    f = ciera.lib().ciera_moe_workspace_bytes
    assert f(-1, 0, 0) == f(0, -1, 0) == f(0, 0, -1) == f(0, 2000, 0) == 0
    base = f(0, 0, 0)
    assert base > 0 and base % 256 == 0
    assert f(10 ** 6, 128, 0) >= base + 10 ** 6 // 64 * 128
    assert f(10 ** 6, 0, 4096) > f(100, 0, 4096) >= base + 4 * 4096
    assert ciera.lib().ciera_moe_workspace_init(None, None) == ciera.E_INVAL
    assert ciera.lib().ciera_moe_workspace_init(vp(4097), None) == ciera.E_INVAL


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.bfloat16)
    for call in (lambda: experts.rmsnorm(x, w), lambda: experts.quantize_rows(x),
                 lambda: experts.rmsnorm_backward(x, x, torch.zeros(4), w),
                 lambda: experts.route(torch.zeros(4, 8), 2),
                 lambda: experts.combine(x, torch.zeros(2, 2, dtype=torch.int32)),
                 lambda: experts.mm(x, torch.zeros(2, 4, 8, dtype=torch.bfloat16),
                                    torch.zeros(3, dtype=torch.int32)),
                 lambda: experts.mm_dx(x, torch.zeros(2, 8, 4, dtype=torch.bfloat16),
                                       torch.zeros(3, dtype=torch.int32)),
                 lambda: experts.mm_dw(x, x, torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="logits"):
        experts.route(torch.zeros(4, 8, dtype=torch.float64), 2)


def test_bucket_views_are_the_workloads_tensors():
    """The views name the same values as the bucket's layout."""
    wl = workloads.workload(2, "experts2")
    bucket = torch.arange(wl.layer_numel, dtype=torch.int64)
    bits = (bucket % 65521).to(torch.int32).to(torch.uint16)
    gate_up, down = experts.bucket_views(bits, 2, 2048, 1024)
    assert gate_up.dtype == torch.bfloat16 and gate_up.shape == (2, 2048, 2048)
    for name, off, n in workloads.layer_offsets(wl):
        e, which = int(name[6:name.index(".")]), name.split(".")[1]
        flat = bits[off:off + n].view(torch.int16)
        got = {"gate": gate_up[e, :1024], "up": gate_up[e, 1024:], "down": down[e]}[which]
        assert torch.equal(got.contiguous().view(-1).view(torch.int16), flat)
    shifted = torch.cat([bits[:5], bits])
    assert torch.equal(experts.bucket_views(shifted, 2, 2048, 1024, 5)[1].view(torch.int16),
                       down.view(torch.int16))
    with pytest.raises(ValueError):
        experts.bucket_views(bits, 3, 2048, 1024)
    with pytest.raises(ValueError):
        experts.bucket_views(bits.view(2, -1), 2, 2048, 1024)


def test_control_block_wants_a_place():
    assert ciera.lib().ciera_moe_control(None) == ciera.E_INVAL


@pytest.mark.parametrize("bad", [dict(ys=7), dict(ys=-8), dict(y=None), dict(y=ODD)])
def test_gather_rows_strided_refuses(bad):
    a = dict(y=FAKE, ys=8)
    a.update(bad)
    assert ciera.lib().ciera_gather_rows_strided(
        vp(FAKE), 8, 3, experts.BF16, None, vp(FAKE), 4, 8, vp(a["y"]), a["ys"], None,
        None) == ciera.E_INVAL
