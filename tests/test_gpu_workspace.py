"""Workspaces of calls captured into graphs, and of calls of several threads."""
import threading

import pytest
import torch

from test_gpu_layers import ffn_inputs, make_ids

pytestmark = pytest.mark.gpu


def steps(lib, ts, ids):
    x, wg, wu, wd, dy = ts
    y, saved = lib.muon_gated_ffn(x, wg, wu, wd, save=True)
    return [y, *lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved), lib.muon_embedding_grad(dy, ids, 20)]


def inputs(tokens, seed):
    return [t.cuda() for t in ffn_inputs(tokens, 64, 200, torch.bfloat16, seed)], make_ids(tokens, 20, seed,
                                                                                            torch.int64).cuda()


def test_graph_keeps_its_workspace(lib):
    """Warmed up and captured on one stream; afterwards a larger eager call
    there, a release of the cached buffers, and new allocations: the replays
    give the eager bits and write over nothing."""
    ts, ids = inputs(70, 1)
    big, big_ids = inputs(3000, 2)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ref = [t.clone() for t in steps(lib, ts, ids)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = steps(lib, ts, ids)
    with torch.cuda.stream(stream):
        steps(lib, big, big_ids)
    torch.cuda.synchronize()
    lib.release_workspace()
    with torch.cuda.stream(stream):
        # what the allocator now hands out on that stream
        fresh = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (1 << 16, 1 << 18, 1 << 20, 1 << 22) * 4]
    torch.cuda.synchronize()
    for _ in range(3):
        for t in outs:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, outs))
        assert all(bool((f == 7).all()) for f in fresh)
        with torch.cuda.stream(stream):
            steps(lib, big, big_ids)


def test_graphs_on_two_streams(lib):
    """Two graphs captured one after the other, replayed on streams of their
    own at the same time."""
    work = [inputs(70 + 30 * k, 3 + k) for k in range(2)]
    ref = [[t.clone() for t in steps(lib, *w)] for w in work]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for w in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([t for _ in range(8) for t in steps(lib, *w)])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for r, o in zip(ref, outs):
            assert all(torch.equal(r[i % len(r)], t) for i, t in enumerate(o))


def test_threads_on_one_stream(lib):
    """Threads that call on the same stream get their own results."""
    work = [inputs(60 + 20 * k, 7 + k) for k in range(4)]
    ref = [[t.clone() for t in steps(lib, *w)] for w in work]
    torch.cuda.synchronize()
    bad = []

    def run(k):
        for _ in range(20):
            got = steps(lib, *work[k])
            if not all(torch.equal(a, b) for a, b in zip(ref[k], got)):
                bad.append(k)
    ts = [threading.Thread(target=run, args=(k,)) for k in range(len(work))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad
