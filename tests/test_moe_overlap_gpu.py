"""Calls that may run at the same time: host threads on one stream, graphs
captured on one stream and replayed on two, a first call made in a capture.
Each has to get its own results."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import moe_reference as ref
from lossless_exponent_reuse_gb300 import ciera, experts
from test_moe_rows_gpu import rand

pytestmark = pytest.mark.gpu
F32 = torch.float32


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def test_scratch_memory_is_each_calls_own():
    s = torch.cuda.current_stream().cuda_stream
    a, b = (experts.workspace(0, s, tokens=500, experts=64, dim=256) for _ in range(2))
    assert a.numel() == b.numel() == ciera.lib().ciera_moe_workspace_bytes(500, 64, 256)
    assert (a.data_ptr() + a.numel() <= b.data_ptr() or b.data_ptr() + b.numel() <= a.data_ptr())
    assert (a == 0).all()


def test_first_calls_made_in_a_capture():
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]))
    code = "import test_moe_overlap_gpu as t; t.first_calls()"
    run = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stderr


def first_calls():
    """A process's first calls, on a stream that has seen none, in a capture: the
    status is set before the graph has run, and a replay gives what plain calls give."""
    tokens, E, k, K, N = 300, 16, 4, 128, 64
    logits, x = rand(tokens, E, seed=40, dtype=F32), rand(tokens, K, seed=41)
    w = rand(E, N, K, seed=42)
    h, weight, rstd = rand(tokens, K, seed=43), rand(K, seed=44), torch.ones(tokens, device="cuda")
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r = experts.route(logits, k)
        y = experts.mm(x, w, r.offsets, tokens=r.tokens)
        dx, dw = experts.rmsnorm_backward(x, h, rstd, weight)
    with torch.cuda.stream(side):
        assert experts.status() == ciera.OK
    for out in (*r, y, dx, dw):
        out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    want = experts.route(logits, k)
    assert same(r, want)
    assert torch.equal(y, experts.mm(x, w, want.offsets, tokens=want.tokens))
    assert same((dx, dw), experts.rmsnorm_backward(x, h, rstd, weight))
    assert experts.status() == ciera.OK


def test_graphs_of_one_capture_stream_replayed_on_two():
    T, E, k, dim = 20000, 128, 8, 512
    inputs, graphs, outs, want = [], [], [], []
    capture = torch.cuda.Stream()
    for i in range(2):
        logits = rand(T, E, seed=50 + i, dtype=F32)
        h, dy, w = (rand(3000, dim, seed=60 + i), rand(3000, dim, seed=70 + i),
                    rand(dim, seed=80 + i))
        rstd = torch.ones(3000, device="cuda")
        inputs.append((logits, h, dy, w, rstd))
        want.append((*experts.route(logits, k), *experts.rmsnorm_backward(dy, h, rstd, w)))
    torch.cuda.synchronize()
    for logits, h, dy, w, rstd in inputs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=capture):
            out = (*experts.route(logits, k), *experts.rmsnorm_backward(dy, h, rstd, w))
        graphs.append(graph)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for out in outs:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
            with torch.cuda.stream(capture):                  # and plain calls beside them
                plain = experts.route(inputs[0][0], k)
        torch.cuda.synchronize()
        assert same(plain, want[0][:5])
        assert same(outs[0], want[0]) and same(outs[1], want[1])


def test_threads_on_one_stream():
    """Two launches of one call stay together, whatever another thread puts between."""
    T, E, k, dim, n = 2000, 64, 8, 256, 4
    logits = [rand(T, E, seed=90 + i, dtype=F32) for i in range(n)]
    rows = [(rand(900, dim, seed=100 + i), rand(900, dim, seed=110 + i), rand(dim, seed=120 + i))
            for i in range(n)]
    rstd = torch.ones(900, device="cuda")
    want = [(*experts.route(l, k), *experts.rmsnorm_backward(dy, h, rstd, w))
            for l, (dy, h, w) in zip(logits, rows)]
    torch.cuda.synchronize()
    wrong, failed = [], []

    def work(i):
        try:
            got = []
            for _ in range(100):
                dy, h, w = rows[i]
                got.append((*experts.route(logits[i], k),
                            *experts.rmsnorm_backward(dy, h, rstd, w)))
            torch.cuda.current_stream().synchronize()
            wrong.extend(i for g in got if not same(g, want[i]))
        except BaseException as e:          # reported by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and not wrong
    assert experts.status() == ciera.OK


def test_products_on_two_streams_share_the_status():
    K, N = 256, 128
    x, w = rand(400, K, seed=130), rand(4, N, K, seed=131)
    offsets = torch.tensor([0, 100, 100, 290, 400], dtype=torch.int32, device="cuda")
    want, size = ref.product(x.double(), w, offsets)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [experts.mm(x, w, offsets, stream=s) for _ in range(10) for s in streams]
    for s in streams:
        assert experts.status(stream=s) == ciera.OK
    for y in got:
        ref.within(y, want, size * (K + 2) * ref.U_F32, "y")
