"""Products whose waits run out: a limit shorter than one contraction ends the
call early.  It has to report that, leave nothing under way, and the next call
has to be right."""
import pytest
import torch

from lossless_exponent_reuse_gb300 import ciera, experts
from test_moe_rows_gpu import rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DEEP = 1 << 20


def offsets_of(*ends):
    return torch.tensor([0, *ends], dtype=torch.int32, device="cuda")


def deep(kind):
    """A call whose contraction takes some milliseconds."""
    if kind == "weights":       # pairs of blocks, groups that end inside a stage
        dy, x = rand(DEEP, 64, seed=1), rand(DEEP, 136, seed=2)
        off = offsets_of(5, DEEP // 2 + 7, DEEP // 2 + 7, DEEP - 3)
        return lambda: experts.mm_dw(dy, x, off, out=torch.empty(4, 64, 136, device="cuda"))
    if kind == "rows":          # pairs of blocks
        dy, w = rand(300, DEEP, seed=3), rand(2, DEEP, 40, seed=4)
        off, pre = offsets_of(33, 290), rand(300, 80, seed=5)
        return lambda: experts.mm_dx(dy, w, off, gated=pre)
    few = kind == "few rows"    # single blocks, rows gathered inside the product
    R = 20 if few else 300
    x, w = rand(40, DEEP, seed=6), rand(2, 80, DEEP, seed=7, scale=0.01)
    off = offsets_of(7, R - 1)
    tokens = torch.arange(R, dtype=torch.int32, device="cuda") % 40
    if kind == "8 bits":
        x, xs = experts.quantize_rows(x)
        w, ws = experts.quantize_rows(w)
        return lambda: experts.mm_gated(x, w, off, tokens=tokens, x_scale=xs, w_scale=ws)
    return lambda: experts.mm_gated(x, w, off, tokens=tokens)


@pytest.mark.parametrize("kind", ["weights", "rows", "many rows", "few rows", "8 bits"])
def test_a_limit_shorter_than_the_contraction(kind):
    call = deep(kind)
    want = call()
    assert experts.status() == ciera.OK
    try:
        for ns in (1, 1000, 5000, 20000, 100000):
            ciera.set_wait_timeout_ns(ns)
            call()
            assert experts.status() == ciera.E_TIMEOUT, ns
            assert experts.status() == ciera.OK          # read once, then cleared
    finally:
        ciera.set_wait_timeout_ns(1_000_000_000)
    assert torch.equal(call(), want)
    assert experts.status() == ciera.OK


def test_a_replayed_graph_reports_to_the_device_s_status():
    """The limit is the one at the time of the capture; whoever asks next hears."""
    call = deep("weights")
    want = call()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    try:
        ciera.set_wait_timeout_ns(1000)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call()
    finally:
        ciera.set_wait_timeout_ns(1_000_000_000)
    assert experts.status() == ciera.OK
    graph.replay()
    assert experts.status() == ciera.E_TIMEOUT
    assert torch.equal(call(), want)
    assert experts.status() == ciera.OK
