"""Attention over the paged cache against its definition in 64 bits: causal
prompts, drafted trees and single tokens, grouped heads, ragged lengths, pages
that end inside a tile, masks that leave rows empty, garbage in places that
nothing sees, and the refusals."""
import numpy as np
import pytest

from cache_common import (Batch, ancestors, attend_bound, attend_exact, compare, dtype, mask_words, random_parents)
from gpu_common import torch_mod

pytestmark = pytest.mark.gpu


def run(w, q, masks=None, words=1, scale=None, lse=False, max_tokens=None, **kw):
    torch = torch_mod()
    out = torch.full(q.shape, 55.0, dtype=q.dtype, device="cuda")
    hq = q.shape[1] if q.dim() == 3 else q.shape[1] // w.head_dim
    ls = torch.full((w.n, hq), 55.0, device="cuda") if lse else None
    tree = None if masks is None else mask_words(masks, words)
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, max(w.tokens) if max_tokens is None else max_tokens,
                   scale=scale, tree=tree, lse=ls, status=w.status, **kw)
    torch.cuda.synchronize()
    return out, ls


def check(w, kv, q64, out, masks=None, scale=None, lse=None, rows=None):
    """Every row (or the listed ones) of every sequence against the definition."""
    hq, d = q64.shape[1], w.head_dim
    scale = d ** -0.5 if scale is None else scale
    seen = w.seen(masks)
    got = out.double().cpu().numpy().reshape(q64.shape)
    assert w.status.cpu().tolist() == [0] * len(w.tokens)
    for b, t in enumerate(w.tokens):
        lo = w.cu_host[b]
        use = np.arange(t) if rows is None else np.array([r for r in rows if r < t], dtype=int)
        if not len(use):
            continue
        s = seen[b][use]
        want, mag, ls, big = attend_exact(q64[lo + use], kv[b], s, scale, hq // w.kv_heads)
        group = hq // w.kv_heads
        vsum = np.einsum("tn,hnd->thd", s.astype(np.float64), np.abs(kv[b][1])).repeat(group, axis=1)
        compare(f"sequence {b}", got[lo + use], want, attend_bound(w.dt, want, mag, big, vsum, d))
        if lse is not None:
            g = lse[lo:lo + t].double().cpu().numpy()[use]
            empty = np.isneginf(ls)
            assert np.array_equal(np.isneginf(g), empty)
            tol = 2 * (d + 4) * 2.0 ** -24 * big + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, ls)))
            compare(f"lse {b}", np.where(empty, 0, g), np.where(empty, 0, ls), tol)


CAUSAL = [
    # tokens, ctx, q_heads, kv_heads, head_dim, page, type
    ([1], [0], 1, 1, 128, 16, "bf16"),
    ([1, 1, 1], [1, 127, 128], 4, 1, 128, 64, "bf16"),
    ([1, 1, 1, 1], [15, 16, 129, 511], 8, 8, 64, 16, "f16"),
    ([2, 0, 7, 1], [0, 5, 120, 0], 8, 2, 128, 32, "f16"),
    ([33, 128, 5], [0, 0, 251], 4, 4, 64, 64, "bf16"),
    ([129, 3], [0, 640], 12, 4, 128, 128, "bf16"),
    ([260], [13], 28, 4, 64, 16, "f16"),
    ([64, 65, 31, 32], [64, 63, 1, 96], 8, 1, 128, 64, "bf16"),
    ([513], [0], 2, 1, 128, 64, "f16"),
    ([300, 7], [300, 1100], 16, 2, 128, 32, "bf16"),
    ([11], [2500], 6, 2, 128, 128, "bf16"),
    ([1] * 40, list(range(0, 800, 20)), 4, 2, 64, 32, "bf16"),
    ([3], [70], 128, 1, 64, 16, "bf16"),
    ([2], [9], 100, 1, 128, 16, "f16"),
]


@pytest.mark.parametrize("case", range(len(CAUSAL)))
def test_causal(tcd, case):
    tokens, ctx, hq, hkv, d, page, dt = CAUSAL[case]
    w = Batch(tcd, tokens, ctx, dt, hkv, d, page, seed=case)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, d)
    out, lse = run(w, q, lse=True)
    check(w, kv, q64, out, lse=lse)


TREES = [
    # tokens, ctx, q_heads, kv_heads, head_dim, page, type, words
    ([1], [0], 1, 1, 64, 16, "bf16", 1),
    ([5, 1, 0, 17], [0, 33, 7, 129], 8, 2, 128, 16, "bf16", 1),
    ([64], [1000], 4, 4, 128, 64, "f16", 1),
    ([37, 9], [91, 1], 16, 2, 64, 32, "bf16", 1),
    ([100, 65, 3], [28, 63, 640], 4, 1, 128, 128, "bf16", 2),
    ([256, 40], [120, 0], 8, 2, 64, 64, "f16", 4),
    ([150], [200], 7, 7, 128, 16, "bf16", 3),
]


@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree(tcd, case):
    tokens, ctx, hq, hkv, d, page, dt, words = TREES[case]
    w = Batch(tcd, tokens, ctx, dt, hkv, d, page, seed=100 + case)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, d)
    masks = [m for n in tokens for m in ancestors(random_parents(w.rng, n))]
    out, lse = run(w, q, masks, words, lse=True)
    check(w, kv, q64, out, masks, lse=lse)


def test_tree_of_one_chain_equals_causal(tcd):
    """The same slots seen through either mask: the same bits."""
    torch = torch_mod()
    w = Batch(tcd, [64, 13], [77, 300], "bf16", 2, 128, 64, seed=7)
    w.fill()
    q, _ = w.normal(w.n, 8, 128)
    masks = [m for n in w.tokens for m in ancestors(list(range(-1, n - 1)))]
    assert torch.equal(run(w, q)[0], run(w, q, masks)[0])


def test_rows_that_see_nothing_are_zero(tcd):
    """No context and an empty mask; bits past the sequence's tokens do not count."""
    w = Batch(tcd, [4, 70], [0, 0], "bf16", 1, 64, 16, seed=1)
    kv = w.fill()
    q, q64 = w.normal(w.n, 3, 64)
    masks = [0, 1 << 4, 0b11, (1 << 63)] + [0 if i % 3 else 1 << (i % 70) for i in range(70)]
    out, lse = run(w, q, masks, 2, lse=True)
    check(w, kv, q64, out, masks, lse=lse)
    host = out.float().cpu().numpy()
    assert not host[[0, 1, 3]].any() and np.isneginf(lse.cpu().numpy()[[0, 1, 3]]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("which", [0, 1])
def test_what_is_not_seen_does_not_count(tcd, bad, which):
    """Infinities and NaN in keys or values of drafted tokens that other
    branches hold, of later tokens of a prompt, of unused slots and pages."""
    torch = torch_mod()
    w = Batch(tcd, [40, 9], [61, 130], "bf16", 2, 128, 16, seed=3)
    kv = w.fill()
    q, q64 = w.normal(w.n, 4, 128)
    trees = [random_parents(w.rng, n) for n in w.tokens]
    masks = [m for t in trees for m in ancestors(t)]
    clean, clean_lse = run(w, q, masks, lse=True)
    causal, _ = run(w, q)
    for b, at in ((0, 20), (1, 4)):
        pages, offs = w.slots(b, w.ctx_list[b] + at, w.ctx_list[b] + at + 1)
        w.pool[0, int(pages[0]), which, :, int(offs[0]), 5:90] = bad
    out, lse = run(w, q, masks, lse=True)
    out2, _ = run(w, q)
    for b, at in ((0, 20), (1, 4)):
        for i in range(w.tokens[b]):
            r = w.cu_host[b] + i
            if not masks[r] >> at & 1:
                assert torch.equal(out[r], clean[r]) and torch.equal(lse[r], clean_lse[r]), (b, i)
            elif which == 1:      # it sees the token: the elements it touches, and no others, go with it
                g = out[r].float()
                assert torch.equal(out[r][:, :5], clean[r][:, :5]) and torch.equal(out[r][:, 90:], clean[r][:, 90:])
                assert (torch.isnan(g[:, 5:90]).all() if bad != bad else (g[:, 5:90] == bad).all()), (b, i)
            elif bad != bad:
                assert torch.isnan(out[r].float()).all(), (b, i)
            if i < at:
                assert torch.equal(out2[r], causal[r]), (b, i)


def test_scores_out_of_range(tcd):
    """Scores of thousands: the largest takes all the weight; of -inf (finite keys, overflowing products): none."""
    torch = torch_mod()
    w = Batch(tcd, [3], [200], "f16", 1, 64, 32, seed=9)
    kv = w.fill(scale=40.0)
    q, q64 = w.normal(w.n, 2, 64)
    q = (q.float() * 40).half()
    q64 = q.double().cpu().numpy()
    out, lse = run(w, q, lse=True)
    check(w, kv, q64, out, lse=lse)
    out, _ = run(w, q, scale=0.0)
    check(w, kv, q64, out, scale=0.0)
    out, _ = run(w, q, scale=-0.3)
    check(w, kv, q64, out, scale=-0.3)


def test_running_maximum_rises_late(tcd):
    """Maxima that grow by any amount from tile to tile, far back and at the end."""
    w = Batch(tcd, [5, 130], [1500, 900], "bf16", 1, 128, 64, seed=11)
    kv = w.fill()
    q, q64 = w.normal(w.n, 4, 128)
    torch = torch_mod()
    for b in range(2):
        n = w.tokens[b] + w.ctx_list[b]
        ramp = torch.linspace(0.01, 3.0, n, device="cuda")
        pages, offs = w.slots(b, 0, n)
        pages, offs = torch.from_numpy(pages).long().cuda(), torch.from_numpy(offs).cuda()
        k = w.pool[0, pages, 0, :, offs].float() * ramp[:, None, None]
        w.pool[0, pages, 0, :, offs] = k.to(w.pool.dtype)
        kv[b][0] = w.pool[0, pages, 0, :, offs].double().cpu().numpy().transpose(1, 0, 2)
    out, lse = run(w, q, lse=True)
    check(w, kv, q64, out, lse=lse, rows=list(range(0, 130, 3)))


def test_strided_rows_and_wider_bounds(tcd):
    """Queries inside a wider projection, outputs inside wider rows, max_tokens larger than needed."""
    torch = torch_mod()
    w = Batch(tcd, [19, 2], [30, 77], "bf16", 2, 64, 16, seed=13)
    kv = w.fill()
    wide, wide64 = w.normal(w.n, 8 * 64 + 40)
    q, q64 = wide[:, 8:8 + 6 * 64], wide64[:, 8:8 + 6 * 64].reshape(w.n, 6, 64)
    buf = torch.full((w.n, 6 * 64 + 16), 55.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, 16:]
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 1000, status=w.status)
    check(w, kv, q64, out)
    assert (buf[:, :16] == 55).all()


def test_each_layer_is_its_own(tcd):
    torch = torch_mod()
    w = Batch(tcd, [4], [50], "f16", 1, 64, 16, layers=3, seed=17)
    kvs = [w.fill(layer) for layer in range(3)]
    q, q64 = w.normal(w.n, 2, 64)
    for layer in (2, 0, 1):
        out = torch.zeros_like(q)
        w.cache.attend(layer, q, w.cu, w.ctx, w.table, out, 4, status=w.status)
        check(w, kvs[layer], q64, out)


def test_repeats_and_batch_composition(tcd):
    """The same call twice gives the same bits."""
    torch = torch_mod()
    w = Batch(tcd, [1, 40, 300, 2], [900, 100, 0, 4000], "bf16", 2, 128, 64, seed=19)
    w.fill()
    q, _ = w.normal(w.n, 8, 128)
    a = run(w, q, lse=True)
    for _ in range(3):
        b = run(w, q, lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_many_sequences(tcd):
    """More sequences than the machine has SMs, most of them short, some empty."""
    rng = np.random.default_rng(2)
    tokens = [int(x) for x in rng.integers(0, 4, 700)]
    ctx = [int(x) for x in rng.integers(0, 200, 700)]
    tokens[5], ctx[5] = 64, 1500
    w = Batch(tcd, tokens, ctx, "bf16", 1, 64, 32, seed=23)
    kv = w.fill()
    q, q64 = w.normal(w.n, 2, 64)
    masks = [m for n in tokens for m in ancestors(random_parents(w.rng, n))]
    out, lse = run(w, q, masks, lse=True)
    check(w, kv, q64, out, masks, lse=lse)


def test_no_tokens(tcd):
    torch = torch_mod()
    w = Batch(tcd, [0, 0], [5, 0], "bf16", 1, 64, 16)
    q = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    run(w, q)
    assert w.status.cpu().tolist() == [0, 0]


def test_other_streams_and_graphs(tcd):
    """On a side stream, inside a captured graph with lengths that change between launches."""
    torch = torch_mod()
    w = Batch(tcd, [2, 3], [500, 60], "bf16", 2, 128, 64, seed=29)
    kv = w.fill()
    q, q64 = w.normal(w.n, 4, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(q)
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 3, status=w.status, stream=side)
    side.synchronize()
    check(w, kv, q64, out)
    ref = out.clone()
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g, stream=side):
        w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 3, status=w.status, stream=side)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    # one cached token fewer: the lengths are read when the graph runs
    w.ctx -= 1
    w.ctx_list = [c - 1 for c in w.ctx_list]
    kv = [x[:, :, :-1] for x in kv]
    g.replay()
    torch.cuda.synchronize()
    check(w, kv, q64, out)


def test_bad_sequences_are_reported(tcd):
    """The others keep their bits."""
    torch = torch_mod()
    w = Batch(tcd, [3, 20, 1, 5], [40, 100, 700, 0], "bf16", 2, 64, 16, seed=31)
    w.fill()
    q, _ = w.normal(w.n, 4, 64)

    def go(max_tokens=20, cu=w.cu, ctx=w.ctx, table=w.table):
        out = torch.full_like(q, 55.0)
        w.cache.attend(0, q, cu, ctx, table, out, max_tokens, status=w.status)
        torch.cuda.synchronize()
        return w.status.cpu().tolist(), out

    st, good = go()
    assert st == [0] * 4
    for bad in (w.pages, -1, 2 ** 31 - 1):
        table = w.table.clone()
        table[1, 3] = bad
        st, out = go(table=table)
        assert st == [0, 19, 0, 0] and torch.equal(out[:3], good[:3]) and torch.equal(out[23:], good[23:])
    st, out = go(max_tokens=19)
    assert st == [0, 19, 0, 0] and torch.equal(out[:3], good[:3]) and torch.equal(out[23:], good[23:])
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        ctx = w.ctx.clone()
        ctx[2] = bad
        st, out = go(ctx=ctx)
        assert st == [0, 0, 19, 0] and torch.equal(out[:23], good[:23]) and torch.equal(out[24:], good[24:])
    for cu, n in (([0, 3, 23, 24, 30], 19), ([0, 3, 23, 22, 29], 0), ([-4, 3, 23, 24, 29], 0)):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        assert 19 in go(cu=cu)[0]


def test_refusals(tcd):
    torch = torch_mod()
    w = Batch(tcd, [2, 1], [3, 4], "bf16", 2, 64, 16)
    w.fill()
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ok = dict(q=q, cu_tokens=w.cu, ctx_lens=w.ctx, page_table=w.table, out=out, max_tokens=2)
    for bad in (dict(q=q.half()), dict(q=q[:, :, :32]), dict(out=out[:2]), dict(out=out.cpu()),
                dict(tree=torch.zeros((3, 1), dtype=torch.int32, device="cuda")),
                dict(tree=torch.zeros((2, 1), dtype=torch.int64, device="cuda")),
                dict(lse=torch.zeros((3, 3), device="cuda")), dict(cu_tokens=w.cu[1:]),
                dict(status=torch.zeros(1, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            w.cache.attend(0, **{**ok, **bad})
    q3 = torch.zeros((3, 3, 64), dtype=torch.bfloat16, device="cuda")
    wide = Batch(tcd, [1], [3], "bf16", 1, 64, 16)
    q129 = torch.zeros((1, 129, 64), dtype=torch.bfloat16, device="cuda")
    words = torch.zeros((3, 5), dtype=torch.int64, device="cuda")
    for call, code in ((lambda: w.cache.attend(0, **{**ok, "q": q3, "out": q3.clone()}), "TC_ERR_UNSUPPORTED"),
                       (lambda: wide.cache.attend(0, q129, wide.cu, wide.ctx, wide.table, q129.clone(), 1),
                        "TC_ERR_UNSUPPORTED"),
                       (lambda: w.cache.attend(0, **{**ok, "tree": words}), "TC_ERR_CAPACITY"),
                       (lambda: w.cache.attend(0, **{**ok, "tree": words[:, :1].contiguous(), "max_tokens": 65}),
                        "TC_ERR_CAPACITY"),
                       (lambda: w.cache.attend(1, **ok), "TC_ERR_INVALID_ARG"),
                       (lambda: w.cache.attend(0, **{**ok, "max_tokens": -1}), "TC_ERR_INVALID_ARG"),
                       (lambda: w.cache.attend(0, **{**ok, "scale": float("nan")}), "TC_ERR_INVALID_ARG")):
        with pytest.raises(tcd.TcError) as e:
            call()
        assert e.value.name == code
    torch.cuda.synchronize()
    assert not out.any()


@pytest.mark.parametrize("shape", [([2, 1], [300, 40]), ([400], [0])])
def test_wait_timeout_is_reported_and_the_next_call_works(tcd, shape):
    """A load that never comes (left out by the test switch): the bounded waits
    run out, the kernel returns, every sequence gets the error; then all is well."""
    w = Batch(tcd, shape[0], shape[1], "bf16", 2, 128, 64, seed=37)
    kv = w.fill()
    q, q64 = w.normal(w.n, 4, 128)
    w.cache.attend_wait_test(True, 2000)
    run(w, q)
    assert w.status.cpu().tolist() == [tcd.TC_ERR_DEVICE_TIMEOUT] * len(w.tokens)
    w.cache.attend_wait_test(False, 0)
    out, _ = run(w, q)
    check(w, kv, q64, out)


def test_long_cache_passes_32_bits(tcd):
    """A pool of more than 2^32 elements, its far end the sequence's pages."""
    torch = torch_mod()
    pages = 300000
    pool = torch.zeros((1, pages, 2, 1, 128, 64), dtype=torch.bfloat16, device="cuda")   # 9.8 GB
    cache = tcd.KvCache(pool)
    n = 1300
    table = torch.tensor([[pages - 1 - 3 * i for i in range(11)]], dtype=torch.int32, device="cuda")
    k = torch.randn((11, 2, 1, 128, 64), device="cuda").bfloat16()
    pool[0, table[0].long()] = k
    flat = k.double().cpu().numpy()[:, :, 0].transpose(1, 0, 2, 3).reshape(2, 1, -1, 64)[:, :, :n]
    q = torch.randn((2, 2, 64), device="cuda").bfloat16()
    out = torch.zeros_like(q)
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([n - 2], dtype=torch.int32, device="cuda")
    cache.attend(0, q, cu, ctx, table, out, 2)
    cache.raise_on_error()
    seen = np.tri(2, n, n - 2, dtype=bool)
    want, mag, _, big = attend_exact(q.double().cpu().numpy(), flat, seen, 0.125, 2)
    compare("out", out.double().cpu().numpy(), want, attend_bound("bf16", want, mag, big, 0.0, 64))
