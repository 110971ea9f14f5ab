"""The attention half over a rebuilt bucket, and its operators run together as a
serving loop runs them: prompts, chunks, single tokens, requests that leave; in
captured graphs, on several streams and from several threads."""
import threading

import pytest
import torch

import attention_reference as ref
from attention_reference import BF16, I32, ints, rand
from lossless_exponent_reuse_gb300 import attention, ciera, experts, moe_layer, workloads
from lossless_exponent_reuse_gb300.allgather import SimulatedAllgather

pytestmark = pytest.mark.gpu


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_heads,heads,dim,page", [(4, 4, 64, 16), (6, 2, 128, 24), (4, 1, 80, 20)])
def test_half_over_a_rebuilt_bucket(q_heads, heads, dim, page, e4m3):
    """Three requests, their prompts in chunks, then single tokens, against causal
    attention over the whole sequences in 64 bits."""
    model = 256
    wl = moe_layer.layer_workload(4, model, 64, ranks=4, block=256, name=f"half{q_heads}{dim}",
                                  attention_rows=(q_heads * dim, heads * dim))
    ag = SimulatedAllgather(wl.numel, wl.block, wl.ranks)
    for w in workloads.sequence(wl, 2):
        rebuilt = ag.step(w.cuda())
    assert ag.status() == ciera.OK
    rotary = attention.rotary_table(dim)
    half = moe_layer.AttentionLayer(rebuilt[:wl.numel], wl, dim, rotary)
    assert half.heads == [q_heads, heads, heads]
    cache = attention.page_cache(60, page, heads, dim, e4m3=e4m3)
    pool = attention.page_pool(60, 3, 30)
    lengths = ints([0, 0, 0])
    xs, ys = [[], [], []], [[], [], []]
    for turn, new in enumerate([[40, 150, 0], [40, 1, 7], [1, 30, 1], [1, 1, 1]]):
        n = sum(new)
        x, residual = rand(n, model, seed=turn), rand(n, model, seed=turn + 50, scale=2.0)
        step = attention.assign_pages(pool, lengths, ints(new), n, page, count=pool.count)
        y, h = half.serve(x, step, cache, residual, longest=max(new))
        assert torch.equal(h, (x.float() + residual.float()).to(BF16))
        lengths = step.lengths
        for r, (a, b) in enumerate(zip(step.offsets.tolist(), step.offsets.tolist()[1:])):
            xs[r].append(x[a:b].double() + residual[a:b].double())
            ys[r].append(y[a:b])
    assert experts.status() == ciera.OK and lengths.tolist() == [82, 182, 9]
    for x, y in zip(xs, ys):
        x, y = torch.cat(x), torch.cat(y)
        normed = x * ((x * x).mean(1, keepdim=True) + half.eps) ** -0.5 * half.norm.double()
        qkv = (normed @ half.qkv.double().T).view(len(x), -1, dim)
        q, k, v = qkv.split(half.heads, 1)
        at = torch.arange(len(x))
        q, k = (ref.rotary(t, at, rotary)[0].cuda() for t in (q, k))
        k, v = (t.repeat_interleave(q_heads // heads, 1) for t in (k, v))
        s = torch.einsum("qhd,khd->hqk", q, k) * dim ** -0.5
        s = s.masked_fill(torch.ones_like(s[0]).triu(1).bool(), float("-inf"))
        o = torch.einsum("hqk,khd->qhd", torch.softmax(s, 2), v)
        want = o.flatten(1) @ half.o.double().T
        # roundings to bf16 of the norm, q, k, v, both products' outputs and the
        # attention's weights and output, 2^-9 each on average, adding up as
        # squares; 8-bit keys and values 2^-5 each
        assert off(y, want) < (8 ** 0.5 * 2.0 ** -9 + 2.0 ** -9 if not e4m3 else 3 * 2.0 ** -5)


def test_half_of_no_tokens():
    wl = moe_layer.layer_workload(2, 128, 64, ranks=1, block=64, name="half_of_none",
                                  attention_rows=(256, 128))
    half = moe_layer.AttentionLayer(rand(wl.numel), wl, 64, attention.rotary_table(64))
    cache = attention.page_cache(4, 16, 2, 64)
    pool = attention.page_pool(4, 2, 2)
    step = attention.assign_pages(pool, ints([0, 0]), ints([0, 0]), 0, 16, count=pool.count)
    y, h = half.serve(rand(0, 128), step, cache)
    assert list(y.shape) == [0, 128] and list(h.shape) == [0, 128]
    assert pool.count.tolist() == [4] and step.offsets.tolist() == [0, 0, 0]
    assert experts.status() == ciera.OK


def small_batch(seed, new, e4m3=False):
    heads, dim, page = 2, 128, 16
    cached = [300, 17, 90]
    cache, table = ref.paged([n + c for n, c in zip(new, cached)], page, heads, dim, seed=seed,
                             e4m3=e4m3)
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    q = rand(off[-1], 4, dim, seed=seed + 9)
    return q, cache, table, ints(off), ints([n + c for n, c in zip(new, cached)])


BATCHES = [(1, [1, 1, 1], False), (2, [200, 5, 64], False), (3, [1, 2, 1], True), (4, [99, 1, 300], True)]


def test_graphs_of_one_capture_stream_replayed_on_two():
    inputs = [small_batch(*b) for b in BATCHES]
    want = [attention.attend(*i) for i in inputs]
    torch.cuda.synchronize()
    capture, graphs, outs = torch.cuda.Stream(), [], []
    for i in inputs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=capture):
            outs.append(attention.attend(*i))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for turn in range(20):
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), turn
    assert experts.status() == ciera.OK


def test_threads_on_one_stream_and_on_their_own():
    inputs = [small_batch(*b) for b in BATCHES]
    # other calls with scratch memory on the same stream
    logits = rand(700, 16, seed=60, dtype=torch.float32)
    h, dy, w = rand(900, 256, seed=61), rand(900, 256, seed=62), rand(256, seed=63)
    rstd = torch.ones(900, device="cuda")
    jobs = [lambda i=i: (attention.attend(*i),) for i in inputs]
    jobs += [lambda: tuple(experts.route(logits, 4)), lambda: experts.rmsnorm_backward(dy, h, rstd, w)]
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    for own in (False, True):
        got = [[] for _ in jobs]
        streams = [torch.cuda.Stream() if own else torch.cuda.current_stream() for _ in jobs]

        def work(at):
            with torch.cuda.stream(streams[at]):
                for _ in range(20):
                    got[at].append(jobs[at]())

        threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
        [t.start() for t in threads]
        [t.join() for t in threads]
        torch.cuda.synchronize()
        for g, expected in zip(got, want):
            assert len(g) == 20
            assert all(torch.equal(a, b) for out in g for a, b in zip(out, expected))
    assert experts.status() == ciera.OK


def test_a_captured_serving_step():
    """A step of single tokens captured once and replayed: lengths, tables, pages and
    caches go on from replay to replay, as the same steps one by one make them."""
    heads, dim, page, R = 2, 128, 16, 3
    rotary = attention.rotary_table(dim)
    both = []
    for captured in (False, True):
        cache = attention.page_cache(40, page, heads, dim)
        pool = attention.page_pool(40, R, 12)
        lengths, new = ints([0] * R), ints([1] * R)
        x = torch.zeros(R, 3 * heads, dim, dtype=BF16, device="cuda")

        def one():
            step = attention.assign_pages(pool, lengths, new, R, page, count=pool.count)
            q, k, v = x.split([heads] * 3, 1)
            q = attention.append(q, k, v, step.positions, step.slots, rotary, cache)
            o = attention.attend(q, cache, pool.table, step.offsets, step.context, longest=1)
            lengths.copy_(step.lengths)
            return o

        outs = []
        if captured:
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                o = one()
        for turn in range(40):
            x.copy_(rand(R, 3 * heads, dim, seed=turn))
            if captured:
                graph.replay()
                outs.append(o.clone())
            else:
                outs.append(one())
        both.append((torch.stack(outs), pool.table.clone(), lengths.clone(), pool.count.clone(),
                     cache.key.clone(), cache.value.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*both))
    assert both[0][2].tolist() == [40] * R and int(both[0][3]) == 40 - R * 3
    assert experts.status() == ciera.OK


def test_on_a_stream_given():
    q, cache, table, off, context = small_batch(*BATCHES[1])
    want = attention.attend(q, cache, table, off, context)
    r, at = attention.rotary_table(128), torch.arange(q.shape[0], device="cuda", dtype=I32)
    turned = attention.rotary(q, at, r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = attention.attend(q, cache, table, off, context, stream=side)
    again = attention.rotary(q, at, r, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(again, turned)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_limit_shorter_than_a_tile(e4m3):
    """Waits that run out: the call ends, says so, leaves nothing under way, and the
    next one is right."""
    q, cache, table, off, context = small_batch(5, [800, 300, 500], e4m3)
    want = attention.attend(q, cache, table, off, context)
    assert experts.status() == ciera.OK
    try:
        for ns in (1, 200, 1000, 5000):
            ciera.set_wait_timeout_ns(ns)
            attention.attend(q, cache, table, off, context)
            torch.cuda.synchronize()
            st = experts.status()
            assert st in (ciera.E_TIMEOUT, ciera.OK), ns
            if ns == 1:
                assert st == ciera.E_TIMEOUT
    finally:
        ciera.set_wait_timeout_ns(10 ** 9)
    assert torch.equal(attention.attend(q, cache, table, off, context), want)
    assert experts.status() == ciera.OK


def test_command_serves_requests(capsys):
    moe_layer.main()
    out = capsys.readouterr().out
    assert out.count("served") == 3 and "FAILED" not in out


def test_layer_refuses_scattered_weights():
    wl = workloads.small("scattered", [(8, 8)] * 3, 1, 8)
    t = [workloads.Tensor(n, (8, 8)) for n in ("attn.q", "attn.v", "attn.k", "attn.o")]
    import dataclasses
    wl = dataclasses.replace(wl, tensors=tuple(t) + (workloads.Tensor("input_norm", (8,)),))
    with pytest.raises(ValueError):
        moe_layer.AttentionLayer(torch.zeros(wl.numel, dtype=BF16), wl, 8,
                                 attention.rotary_table(8, device="cpu"))
