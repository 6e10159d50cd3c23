"""That calls of tc_attend_shared go the way that they are meant to: contexts that are
small together are read sequence by sequence, others share their prefix; and a layer's
step, forked pages and workspaces that grow on the sharing side, with tables wide
enough for it.  What only the sharing way writes is the part of the workspace behind
tc_attend's."""
import numpy as np
import pytest

import test_gpu_layer as layer
from gpu_common import torch_mod
from test_gpu_attend_shared import CASES, LONG, MANY, Groups, build, many

pytestmark = pytest.mark.gpu


def pages_to_share(batch, rows, page, kv_heads, head_dim):
    """Pages of a table that leave no doubt: the rule's border is 16 MB, and 4 MB for each row of a sequence."""
    return ((20 << 20) + (5 << 20) * rows) // (batch * page * kv_heads * head_dim * 4) + 1


def widen(table, width):
    torch = torch_mod()
    more = torch.full((table.shape[0], max(0, width - table.shape[1])), -1, dtype=table.dtype, device=table.device)
    return torch.cat((table, more), 1).contiguous()


def shares(cache, q, cu, ctx, table, max_tokens, cu_seqs, lens):
    torch = torch_mod()
    flat = q.view(q.shape[0], -1)
    heads = flat.shape[1] // cache.head_dim
    ws = torch.full((cache.shared_workspace_bytes(q.shape[0], heads),), 0x5a, dtype=torch.uint8, device="cuda")
    status = torch.zeros(table.shape[0], dtype=torch.int32, device="cuda")
    cache.attend_shared(0, q, cu, ctx, table, torch.empty_like(q), max_tokens, cu_seqs, lens, workspace=ws, status=status)
    assert not status.any()
    return bool((ws[cache.workspace_bytes - 1024:] != 0x5a).any())   # (tc_attend leaves the last 1.8 KB of its own alone)


def of(w, q):
    return shares(w.cache, q, w.cu, w.ctx, w.table, max(w.tokens), w.cu_seqs, w.shared)


@pytest.mark.parametrize("room", [17, 0])
def test_batches_of_the_other_tests(tcd, room):
    """Those with room share, where two sequences have a page in common; those without do not."""
    for i, case in enumerate(CASES):
        w, hq = build(tcd, case, i, room)
        w.fill()
        if room == 0 and i in (4, 12):
            continue                                  # (contexts that are not small by themselves)
        common = any(hi - lo > 1 and shared // w.page for lo, hi, shared in w.groups)
        assert of(w, w.normal(w.n, hq, w.head_dim)[0]) == (common and room > 0), i


def test_many_and_long_batches(tcd):
    for i in range(len(MANY)):
        w, hq = many(tcd, i, 60 + i)
        w.fill()
        assert of(w, w.normal(w.n, hq, w.head_dim)[0]), i
    for batch, group, hkv, d, page, dt, prefix in LONG:
        w = Groups(tcd, [1] * batch, [prefix] * batch, [(0, batch, prefix)], dt, hkv, d, page, 1, heads=group)
        w.fill()
        assert of(w, w.normal(w.n, group * hkv, d)[0])


class Wide(layer.Step):
    """A layer's step whose tables have room for long contexts."""

    def __init__(self, tcd, dt, batch):
        super().__init__(tcd, dt, batch)
        self.table = widen(self.table, pages_to_share(batch, layer.HQ // layer.HKV, layer.PAGE, layer.HKV, layer.D))
        q = self.normal(batch, layer.HQ, layer.D)
        assert shares(self.cache, q, self.cu, self.ctx, self.table, 1, *self.groups)


@pytest.fixture
def wide(monkeypatch):
    monkeypatch.setattr(layer, "Step", Wide)


@pytest.mark.parametrize("batch", [3, 90])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_step(tcd, dt, batch, wide):
    layer.test_step(tcd, dt, batch)


def test_step_in_a_graph_beside_plain_calls(tcd, wide):
    layer.test_step_in_a_graph_beside_plain_calls(tcd)


def test_calls_on_a_stream_that_is_not_the_current_one(tcd, wide):
    layer.test_calls_on_a_stream_that_is_not_the_current_one(tcd)


@pytest.mark.parametrize("sequences", [3, 40])
@pytest.mark.parametrize("share", [True, False])
def test_forked_pages(tcd, share, sequences):
    """The pages that a pool hands out: a prompt is forked, the last, partly filled page is copied on its first write."""
    torch = torch_mod()
    page, prompt, n, hq, hkv, d = 16, 37, sequences, 8, 2, 64
    pool = tcd.PagePool(8 + 2 * n, page)
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = tcd.KvCache(torch.randn((1, 8 + 2 * n, 2, hkv, page, d), generator=g, device="cuda").bfloat16())
    seqs = [pool.open()]
    pool.reserve(seqs[0], 0, prompt)
    seqs += [pool.fork(seqs[0], prompt) for _ in range(n - 1)]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for s in seqs:
        for a, b in pool.reserve(s, prompt, prompt + 1):
            cache.copy_pages(ints([a]), ints([b]))
    table = ints(np.stack([pool.row(s, 4) for s in seqs]))
    if share:
        table = widen(table, pages_to_share(n, hq // hkv, page, hkv, d))
    ctx, cu, groups = ints([prompt] * n), ints(list(range(n + 1))), (ints([0, n]), ints([prompt]))
    q = torch.randn((n, hq, d), generator=g, device="cuda").bfloat16()
    assert shares(cache, q, cu, ctx, table, 1, *groups) == share
    out, plain = torch.empty_like(q), torch.empty_like(q)
    cache.attend_shared(0, q, cu, ctx, table, out, 1, *groups)
    cache.attend(0, q, cu, ctx, table, plain, 1)
    cache.raise_on_error()
    # two results of the same sums, in other orders: each within its weights' and its output's roundings
    v = cache.pool[0, :, 1].float().abs().max().item()
    assert float((out.float() - plain.float()).abs().max()) <= 4 * 2.0 ** -8 * v


def test_workspaces_grow_with_calls_and_graphs(tcd):
    """Calls of more and more tokens on one object, in one graph, in graphs side by side and beside plain calls: all
    share, the last one with a kernel for short rests."""
    torch = torch_mod()
    big, hq = build(tcd, ([1] * 100, [9] * 100, [(0, 100, 512)], 8, 2, 128, 64, "bf16"), 5)
    big.fill()
    q, _ = big.normal(100, hq, 128)
    sizes = (2, 17, 100)
    edges = {n: torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in sizes}
    table = {n: widen(big.table[:n], pages_to_share(n, 4, 64, 2, 128)) for n in sizes}
    for n in sizes:
        assert shares(big.cache, q[:n], big.cu[:n + 1], big.ctx[:n], table[n], 1, edges[n], big.shared)

    def call(n, out, stream=None):
        """The first n sequences."""
        big.cache.attend_shared(0, q[:n], big.cu[:n + 1], big.ctx[:n], table[n], out, 1, edges[n], big.shared,
                                stream=stream)

    want = {n: torch.empty_like(q[:n]) for n in sizes}
    for n in sizes:
        call(n, want[n])
    big.cache.raise_on_error()
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for s, order in zip(streams, (sizes, sizes[::-1])):
        g = torch.cuda.CUDAGraph()
        got = {n: torch.zeros_like(want[n]) for n in sizes}
        with torch.cuda.graph(g, stream=s):
            for n in order:
                call(n, got[n])
        graphs.append(g)
        outs.append(got)
    beside = {n: torch.zeros_like(want[n]) for n in sizes}
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        for n in sizes:
            call(n, beside[n], streams[2])
    big.cache.raise_on_error()
    for got in outs + [beside]:
        for n in sizes:
            assert torch.equal(got[n], want[n])
