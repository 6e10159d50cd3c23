"""Captured calls and calls on several streams of one cache object (GPU): what
they use is not shared, and stays as long as the graph."""
import gc
import time

import pytest

from cache_common import Batch
from gpu_common import torch_mod

pytestmark = pytest.mark.gpu


class Work:
    """One batch whose items are cut over workers, on a cache that others use too."""

    def __init__(self, tcd, tokens, ctx, seed):
        torch = torch_mod()
        self.w = Batch(tcd, tokens, ctx, "bf16", 2, 128, 64, seed=seed)
        self.w.fill()
        self.q, _ = self.w.normal(self.w.n, 8, 128)
        self.out = torch.zeros_like(self.q)

    def run(self, **kw):
        w = self.w
        w.cache.attend(0, self.q, w.cu, w.ctx, w.table, self.out, max(w.tokens), **kw)


def pair(tcd):
    """Two batches of different lengths over one pool and one KvCache."""
    torch = torch_mod()
    a = Work(tcd, [300, 2], [5000, 9000], 1)
    b = Work(tcd, [1, 3, 700], [12000, 400, 1000], 2)
    pool = torch.cat((a.w.pool, b.w.pool), 1)
    b.w.table += a.w.pages
    a.w.cache = b.w.cache = tcd.KvCache(pool)
    for x in (a, b):
        x.run()
        torch.cuda.synchronize()
        x.want = x.out.clone()
        x.out.zero_()
    a.w.cache.raise_on_error()
    return a, b


def captured(x, **kw):
    torch = torch_mod()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, **kw):
        for _ in range(3):
            x.run()
    return g


def test_graphs_captured_on_one_stream_run_side_by_side(tcd):
    torch = torch_mod()
    a, b = pair(tcd)
    graphs = captured(a), captured(b)
    cache = a.w.cache
    assert len({o.place[0] for o in (*cache._captured.values(), *cache._own.values())}) == 3
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        for x in (a, b):
            x.out.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(4):
                    g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, a.want) and torch.equal(b.out, b.want)
    cache.raise_on_error()


def test_a_replay_beside_calls_on_the_capture_stream(tcd):
    torch = torch_mod()
    a, b = pair(tcd)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.run()
    torch.cuda.synchronize()
    g = captured(a, stream=side)
    for _ in range(10):
        for x in (a, b):
            x.out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            for _ in range(4):
                g.replay()
        with torch.cuda.stream(side):
            for _ in range(12):
                b.run()
        torch.cuda.synchronize()
        assert torch.equal(a.out, a.want) and torch.equal(b.out, b.want)


def test_two_streams_at_once(tcd):
    torch = torch_mod()
    a, b = pair(tcd)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        for x in (a, b):
            x.out.zero_()
        torch.cuda.synchronize()
        for _ in range(8):
            a.run(stream=streams[0])
            b.run(stream=streams[1])
        torch.cuda.synchronize()
        assert torch.equal(a.out, a.want) and torch.equal(b.out, b.want)
    a.w.cache.raise_on_error()


def test_a_graph_outlives_the_cache_object(tcd):
    """Its buffers are not handed out again while it exists, and are given back after it."""
    torch = torch_mod()
    a, b = pair(tcd)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a.run()
    torch.cuda.synchronize()
    g = captured(a, stream=side)
    own = next(iter(a.w.cache._captured.values()))
    codes, space = own.codes.codes, own.workspace
    mine = {codes.data_ptr(), space.data_ptr()}
    sizes = codes.numel(), space.numel() // 4
    del codes, space
    pool = a.w.cache.pool                             # (the caller's)
    a.w.cache = b.w.cache = None
    gc.collect()
    fill = []
    for s in (torch.cuda.current_stream(), side, torch.cuda.ExternalStream(own.stream)):
        with torch.cuda.stream(s):
            fill += [torch.full((n,), 7, dtype=torch.int32, device="cuda") for n in sizes for _ in range(6)]
    torch.cuda.synchronize()
    assert not mine & {t.data_ptr() for t in fill}
    a.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, a.want) and all(bool((t == 7).all()) for t in fill)
    assert any(o is own for o in tcd._held) and not own.idle()
    g.reset()
    del g
    gc.collect()
    torch.cuda.synchronize()
    end = time.time() + 5
    while not own.idle() and time.time() < end:
        time.sleep(0.01)
    assert own.idle()
    del pool


def test_errors_of_a_graph_stay_until_they_are_raised(tcd):
    """Codes that no call outside a capture has touched."""
    torch = torch_mod()
    x = Work(tcd, [3, 2], [70, 10], 5)
    g = captured(x)
    good = x.w.ctx.clone()
    g.replay()
    x.w.cache.raise_on_error()
    x.w.ctx[1] = -1
    g.replay()
    x.w.ctx.copy_(good)
    g.replay()
    with pytest.raises(tcd.TcError) as e:
        x.w.cache.raise_on_error()
    assert e.value.name == "TC_ERR_BOUNDS" and "sequence 1" in str(e.value)
    g.replay()
    x.w.cache.raise_on_error()


def test_a_workspace_of_the_caller(tcd):
    torch = torch_mod()
    a, _ = pair(tcd)
    cache = a.w.cache
    own = torch.zeros(cache.workspace_bytes, dtype=torch.uint8, device="cuda")
    a.run(workspace=own)
    assert torch.equal(a.out, a.want) and bool(own.any())
    st = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(workspace=own, status=st)
    assert not cache._captured                        # (nothing of the object is used)
    a.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, a.want) and st.tolist() == [0, 0]
    for bad in (own[::2], own.cpu()):
        with pytest.raises(ValueError):
            a.run(workspace=bad)
    for bad in (own[:-1], torch.zeros(cache.workspace_bytes + 8, dtype=torch.uint8, device="cuda")[8:]):
        with pytest.raises(tcd.TcError) as e:
            a.run(workspace=bad)
        assert e.value.name == "TC_ERR_CAPACITY"
