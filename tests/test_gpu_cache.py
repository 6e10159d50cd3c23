"""Append, page copies, compaction and tree masks of the paged cache against
their definitions in 64 bits, and their refusals."""
import ctypes

import numpy as np
import pytest

from cache_common import UNIT, Batch, ancestors, compare, dtype, random_parents
from gpu_common import torch_mod

pytestmark = pytest.mark.gpu


def bits(t):
    torch = torch_mod()
    return t.contiguous().view(torch.int16).cpu().numpy()


def append_exact(x, weight, eps, rot, interleaved):
    """Norm, weight and rotation of heads [n, heads, d] in 64 bits; rot [n, d / 2, 2] or None."""
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    if rot is None:
        return x, np.abs(x)
    d = x.shape[-1]
    first = np.arange(d // 2) * 2 if interleaved else np.arange(d // 2)
    second = first + (1 if interleaved else d // 2)
    a, b = x[..., first], x[..., second]
    c, s = rot[:, None, :, 0], rot[:, None, :, 1]
    y, mag = np.empty_like(x), np.empty_like(x)
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    mag[..., first], mag[..., second] = abs(a * c) + abs(b * s), abs(b * c) + abs(a * s)
    return y, mag


APPENDS = [
    # tokens, ctx, q_heads, kv_heads, head_dim, page, type, norm, rope, interleaved, sliced rows
    ([1], [0], 1, 1, 128, 16, "bf16", True, True, False, False),
    ([1], [777], 16, 4, 128, 64, "bf16", True, True, False, True),
    ([1, 0, 3, 1], [5, 9, 0, 15], 8, 2, 64, 16, "f16", True, True, True, False),
    ([130, 1, 64], [0, 31, 32], 6, 2, 64, 32, "bf16", True, True, True, True),
    ([17, 300], [100, 3], 28, 4, 128, 128, "f16", True, True, False, False),
    ([40], [8], 5, 5, 128, 16, "bf16", False, True, False, False),
    ([40], [8], 4, 1, 64, 16, "bf16", True, False, False, False),
    ([9, 8], [7, 8], 3, 1, 64, 16, "f16", False, False, False, True),
    ([2] * 70 + [0, 41], list(range(70)) + [3, 0], 7, 1, 128, 16, "bf16", True, True, False, False),
]


@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(tcd, case):
    torch = torch_mod()
    tokens, ctx, hq, hkv, d, page, dt, norm, rope, inter, sliced = APPENDS[case]
    eps = 1e-5
    w = Batch(tcd, tokens, ctx, dt, hkv, d, page, layers=2, seed=case)
    before = bits(w.pool).copy()
    cols = (hq + 2 * hkv) * d
    qkv, x = w.normal(w.n, cols + (24 if sliced else 0))
    qkv, x = qkv[:, :cols], x[:, :cols].reshape(w.n, hq + 2 * hkv, d)
    q_out = torch.zeros((w.n, hq * d + (16 if sliced else 0)), dtype=dtype(dt), device="cuda")[:, :hq * d]
    qw, qw64 = w.normal(d) if norm else (None, None)
    kw, kw64 = w.normal(d) if norm else (None, None)
    rot = pos = rope_t = None
    if rope:
        table = w.rng.uniform(-1, 1, (900, d // 2, 2)).astype(np.float32)   # any pairs: the operator only multiplies
        rope_t = torch.from_numpy(table).cuda()
        slot = np.concatenate([np.arange(t) + c for t, c in zip(tokens, ctx)])
        if case % 2:
            p = w.rng.integers(0, 900, w.n).astype(np.int32)
            pos = torch.from_numpy(p).cuda()
        else:
            p = slot
        rot = table[p].astype(np.float64)
    w.cache.append(1, qkv, w.cu, w.ctx, w.table, q_out, q_weight=qw, k_weight=kw, eps=eps, rope=rope_t, positions=pos,
                   interleaved=inter, status=w.status)
    torch.cuda.synchronize()
    assert w.status.cpu().tolist() == [0] * len(tokens)
    # An element is a sum of two products of a norm (d squares, a root, two
    # factors) and an angle, in 32 bits, and is rounded once.
    u = UNIT[dt]

    def check(what, got, heads, weight):
        want, mag = append_exact(heads, weight, eps, rot, inter)
        err = (d + 10) * 2.0 ** -24 * mag
        compare(what, got, want, err + u * (np.abs(want) + err) + 2.0 ** -25)

    check("q", q_out.double().cpu().numpy().reshape(w.n, hq, d), x[:, :hq], qw64)
    after = bits(w.pool).copy()
    pool = w.pool[1].double().cpu().numpy()
    rows = []
    for b, (t, c) in enumerate(zip(tokens, ctx)):
        pages, offs = w.slots(b, c, c + t)
        rows += list(zip(pages, offs))
    rows = np.array(rows).reshape(-1, 2)
    check("k", pool[rows[:, 0], 0, :, rows[:, 1]], x[:, hq:hq + hkv], kw64)
    assert np.array_equal(pool[rows[:, 0], 1, :, rows[:, 1]], x[:, hq + hkv:])
    # nothing else of the pool changed
    after[1][rows[:, 0], :, :, rows[:, 1]] = before[1][rows[:, 0], :, :, rows[:, 1]]
    assert np.array_equal(after, before)


def test_append_reports_bad_sequences_and_leaves_the_rest(tcd):
    torch = torch_mod()
    w = Batch(tcd, [3, 4, 5, 2], [0, 20, 7, 40], "bf16", 1, 64, 16, seed=5)
    qkv, _ = w.normal(w.n, 3 * 64)
    rope = torch.ones((43, 32, 2), device="cuda")

    def run(cu=w.cu, ctx=w.ctx, table=w.table, pos=None):
        w.pool.fill_(float("nan"))
        q = torch.full((w.n, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        w.cache.append(0, qkv, cu, ctx, table, q, rope=rope, positions=pos, status=w.status)
        torch.cuda.synchronize()
        return w.status.cpu().tolist(), q

    ok, good = run()
    assert ok == [0, 0, 0, 0]
    for bad in (10 ** 6, w.pages, -1):
        table = w.table.clone()
        table[2, 0] = bad                      # slots 7..11 of sequence 2
        st, q = run(table=table)
        assert st == [0, 0, 19, 0]
        assert torch.equal(q[:7], good[:7]) and torch.equal(q[12:], good[12:])
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        ctx = w.ctx.clone()
        ctx[1] = bad
        assert run(ctx=ctx)[0] == [0, 19, 0, 0]
    for cu, want in (([0, 3, 7, 12, 15], [0, 0, 0, 19]), ([0, 3, 2, 12, 14], [0, 19, 0, 0]),
                     ([-2, 3, 7, 12, 14], [19, 0, 0, 0])):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        got = run(cu=cu)[0]
        assert [g for g, x in zip(got, want) if x] == [19] and got[0] in (0, 19)
    pos = torch.zeros(w.n, dtype=torch.int32, device="cuda")
    pos[13] = 43
    assert run(pos=pos)[0] == [0, 0, 0, 19]
    pos[13] = -1
    assert run(pos=pos)[0] == [0, 0, 0, 19]
    st = w.status
    w.status = None
    w.cache.append(0, qkv, w.cu, ctx, w.table, good)
    with pytest.raises(tcd.TcError) as e:
        w.cache.raise_on_error()
    assert e.value.name == "TC_ERR_BOUNDS"
    w.status = st


@pytest.mark.parametrize("n,layers,kv_heads,page,d,dt", [
    (1, 1, 1, 16, 64, "bf16"), (5, 3, 2, 128, 128, "f16"), (33, 2, 3, 16, 64, "bf16")])
def test_copy_pages(tcd, n, layers, kv_heads, page, d, dt):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(n)
    raw = torch.randint(-32768, 32768, (layers, 2 * n + 3, 2, kv_heads, page, d), generator=g, device="cuda",
                        dtype=torch.int16)
    pool = raw.clone().view(dtype(dt))             # any bits, NaN among them
    order = torch.randperm(2 * n + 3, generator=g, device="cuda").to(torch.int32)
    src, dst = order[:n].contiguous(), order[n:2 * n].contiguous()
    status = torch.full((n,), 7, dtype=torch.int32, device="cuda")
    tcd.KvCache(pool).copy_pages(src, dst, status=status)
    want = raw.clone()
    want[:, dst.long()] = raw[:, src.long()]
    assert torch.equal(pool.view(torch.int16), want) and status.cpu().tolist() == [0] * n


def test_copy_pages_refuses_bad_ids(tcd):
    torch = torch_mod()
    pool = torch.randn((2, 5, 2, 1, 16, 64), device="cuda").half()
    want = pool.clone()
    want[:, 4] = pool[:, 0]
    src = torch.tensor([5, 0, 1, -1], dtype=torch.int32, device="cuda")
    dst = torch.tensor([2, 4, 7, 3], dtype=torch.int32, device="cuda")
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    cache = tcd.KvCache(pool)
    cache.copy_pages(src, dst, status=st)
    assert st.cpu().tolist() == [19, 0, 19, 19] and torch.equal(pool, want)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    cache.copy_pages(none, none)


@pytest.mark.parametrize("layers,kv_heads,page,d,dt,seed", [
    (1, 1, 16, 64, "bf16", 0), (3, 2, 16, 128, "f16", 1), (2, 5, 64, 64, "bf16", 2), (1, 8, 128, 128, "bf16", 3)])
def test_compact(tcd, layers, kv_heads, page, d, dt, seed):
    """Paths that overlap their own sources, cross pages, keep everything, move nothing."""
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    tokens = [1, 40, 17, 256, 64, 9, 0, 30]
    ctx = [0, 3, 15, 100, 16, 0, 5, 31]
    w = Batch(tcd, tokens, ctx, dt, kv_heads, d, page, layers=layers, seed=seed)
    paths = [[0], sorted(rng.choice(40, 11, replace=False)), list(range(17)), sorted(rng.choice(256, 100, replace=False)),
             [63], [], [], list(range(1, 30))]
    raw = torch.randint(-32768, 32768, tuple(w.pool.shape), device="cuda", dtype=torch.int16)
    w.pool.view(torch.int16).copy_(raw)
    wide = max(len(p) for p in paths)
    path = torch.full((8, wide), -9, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor([int(x) for x in p], dtype=torch.int32)
    n = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
    lens = torch.zeros(8, dtype=torch.int32, device="cuda")
    w.cache.compact(w.table, w.ctx, path.cuda(), n, lens, status=w.status)
    want = raw.cpu().numpy().copy()
    old = raw.cpu().numpy()
    for b, p in enumerate(paths):
        for i, x in enumerate(p):
            (fp,), (fo,) = w.slots(b, ctx[b] + x, ctx[b] + x + 1)
            (tp,), (to,) = w.slots(b, ctx[b] + i, ctx[b] + i + 1)
            want[:, tp, :, :, to] = old[:, fp, :, :, fo]
    assert w.status.cpu().tolist() == [0] * 8
    assert lens.cpu().tolist() == [c + len(p) for c, p in zip(ctx, paths)]
    assert np.array_equal(w.pool.view(torch.int16).cpu().numpy(), want)


def test_compact_reports_bad_paths(tcd):
    torch = torch_mod()
    w = Batch(tcd, [8] * 7, [4] * 7, "bf16", 1, 64, 16, seed=3, extra_width=0)
    w.fill()
    before = bits(w.pool)
    path = torch.tensor([[1, 1, 0], [0, -1, 0], [2, 3, 28], [1, 2, 3], [1, 2, 3], [-1, 0, 1], [1, 2, 3]],
                        dtype=torch.int32, device="cuda")
    n = torch.tensor([2, 2, 3, 4, -1, 2, 2], dtype=torch.int32, device="cuda")
    lens = torch.zeros(7, dtype=torch.int32, device="cuda")
    table = w.table.clone()
    table[6, 0] = w.pages
    w.cache.compact(table, w.ctx, path, n, lens, status=w.status)
    assert w.status.cpu().tolist() == [19] * 7 and lens.cpu().tolist() == [4] * 7
    assert np.array_equal(bits(w.pool), before)


@pytest.mark.parametrize("words", [1, 2, 3, 4])
def test_tree_masks(tcd, words):
    torch = torch_mod()
    rng = np.random.default_rng(words)
    tokens = [1, 0, 64 * words, 37, 64 * words - 1, 5]
    ctx = [0, 4, 1000, 3, 77, 12]
    trees = [random_parents(rng, n) for n in tokens]
    trees[2] = list(range(-1, 64 * words - 1))         # one chain, every bit
    parents = torch.tensor([p for t in trees for p in t], dtype=torch.int32, device="cuda")
    cu = torch.tensor(np.concatenate(([0], np.cumsum(tokens))), dtype=torch.int32, device="cuda")
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    masks = torch.full((len(parents), words), 5, dtype=torch.int64, device="cuda")
    pos = torch.zeros(len(parents), dtype=torch.int32, device="cuda")
    st = tcd.tree_masks(parents, cu, c, masks, pos)
    assert st.cpu().tolist() == [0] * 6
    got = masks.cpu().numpy().view(np.uint64)
    i = 0
    for t, base in zip(trees, ctx):
        for m in ancestors(t):
            assert sum(int(x) << 64 * k for k, x in enumerate(got[i])) == m
            assert int(pos[i]) == base + bin(m).count("1") - 1
            i += 1


def test_tree_masks_reports_bad_parents(tcd):
    torch = torch_mod()
    cu = torch.tensor([0, 2, 4, 6, 71, 72, 80], dtype=torch.int32, device="cuda")
    parents = torch.tensor([-1, 0, -1, 1, -2, 0] + [-1] * 65 + [-1] + [0] * 7, dtype=torch.int32, device="cuda")
    ctx = torch.tensor([1, 1, 1, 1, 1, 1], dtype=torch.int32, device="cuda")
    masks = torch.full((len(parents), 1), 5, dtype=torch.int64, device="cuda")
    st = tcd.tree_masks(parents, cu, ctx, masks)
    # token 1 its own parent; parent -2; 65 tokens in one word; rows past the arrays
    assert st.cpu().tolist() == [0, 19, 19, 19, 0, 19]
    assert masks[:2, 0].cpu().tolist() == [1, 3] and not masks[2:71].any() and masks[71, 0].item() == 1


def test_refusals(tcd):
    """Wrong arguments are refused at once, with a message, and launch nothing."""
    torch = torch_mod()
    for shape in ((1, 4, 2, 1, 16), (1, 4, 3, 1, 16, 64)):
        with pytest.raises(ValueError):
            tcd.KvCache(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        tcd.KvCache(torch.zeros((1, 4, 2, 1, 16, 64), device="cuda"))
    with pytest.raises(ValueError):
        tcd.KvCache(torch.zeros((1, 4, 2, 1, 16, 64), dtype=torch.bfloat16))
    for shape in ((1, 4, 2, 1, 16, 96), (1, 4, 2, 1, 24, 64), (1, 4, 2, 1, 256, 64)):
        with pytest.raises(tcd.TcError) as e:
            tcd.KvCache(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))
        assert e.value.name == "TC_ERR_UNSUPPORTED"
    w = Batch(tcd, [2, 1], [3, 4], "bf16", 2, 64, 16)
    before = bits(w.pool)
    qkv, _ = w.normal(3, 8 * 64)
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    ok = dict(qkv=qkv, cu_tokens=w.cu, ctx_lens=w.ctx, page_table=w.table, q_out=q)
    rope = torch.zeros((9, 32, 2), device="cuda")
    for bad in (dict(qkv=qkv[:, :7 * 64]), dict(qkv=qkv.half()), dict(qkv=qkv.cpu()), dict(qkv=qkv.t()),
                dict(cu_tokens=w.cu.long()), dict(cu_tokens=w.cu[:2]), dict(ctx_lens=w.ctx.cpu()),
                dict(page_table=w.table[:1]), dict(q_out=q[:2]), dict(q_out=q.float()), dict(rope=rope[..., 0]),
                dict(rope=rope.double()), dict(positions=torch.zeros(2, dtype=torch.int32, device="cuda")),
                dict(q_weight=torch.zeros(64, device="cuda")), dict(k_weight=q[0, 0, :32]),
                dict(status=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            w.cache.append(0, **{**ok, **bad})
    for layer in (-1, 1):
        with pytest.raises(tcd.TcError) as e:
            w.cache.append(layer, **ok)
        assert e.value.name == "TC_ERR_INVALID_ARG"
    odd = torch.zeros(3 * 8 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(3, 8 * 64)
    for bad in (dict(qkv=odd), dict(qkv=torch.zeros((3, 8 * 64 + 4), dtype=torch.bfloat16, device="cuda")[:, :8 * 64])):
        with pytest.raises(tcd.TcError) as e:
            w.cache.append(0, **{**ok, **bad})
        assert e.value.name == "TC_ERR_INVALID_ARG"
    path, n = torch.zeros((2, 1), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    with pytest.raises(tcd.TcError) as e:
        w.cache.compact(w.table, w.ctx, path, n, w.ctx)
    assert e.value.name == "TC_ERR_INVALID_ARG"
    with pytest.raises(tcd.TcError) as e:
        w.cache.compact(w.table, w.ctx, torch.zeros((2, 257), dtype=torch.int32, device="cuda"), n, n.clone())
    assert e.value.name == "TC_ERR_CAPACITY"
    with pytest.raises(tcd.TcError):
        tcd.tree_masks(path[:, 0].contiguous(), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), n,
                       torch.zeros((2, 5), dtype=torch.int64, device="cuda"))
    # the C calls refuse NULL as well
    null = ctypes.c_void_p()
    assert tcd._kv_append(None, 0, None, None, None, null) == 1
    assert tcd._kv_append(w.cache._kvp, 0, None, None, None, null) == 1
    assert tcd._attend(w.cache._kvp, 0, None, None, None, 0, None, null) == 1
    assert tcd._kv_copy_pages(w.cache._kvp, None, None, 3, None, null) == 1
    assert tcd._kv_compact(w.cache._kvp, None, None, 1, None, None, None, null) == 1
    assert tcd._tree_masks(None, None, 1, None, None, None, null) == 1
    torch.cuda.synchronize()
    assert np.array_equal(bits(w.pool), before)


def test_long_cache_passes_32_bits(tcd):
    """A pool of more than 2^32 bytes: appends, copies and compaction at its far end."""
    torch = torch_mod()
    pages = 140000                                  # 140000 pages of 32 KiB: 4.6 GB
    pool = torch.zeros((1, pages, 2, 1, 128, 64), dtype=torch.float16, device="cuda")
    cache = tcd.KvCache(pool)
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([126], dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    qkv = torch.randn((3, 3 * 64), device="cuda").half()
    q = torch.zeros((3, 64), dtype=torch.float16, device="cuda")
    cache.append(0, qkv, cu, ctx, table, q)
    assert torch.equal(q, qkv[:, :64])
    kv = qkv[:, 64:].view(3, 2, 64)
    assert torch.equal(pool[0, pages - 1, :, 0, 126:], kv[:2].transpose(0, 1))
    assert torch.equal(pool[0, pages - 2, :, 0, 0], kv[2])
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.compact(table, ctx, torch.tensor([[2]], dtype=torch.int32, device="cuda"),
                  torch.tensor([1], dtype=torch.int32, device="cuda"), lens)
    assert torch.equal(pool[0, pages - 1, :, 0, 126], kv[2]) and lens.item() == 127
    cache.copy_pages(torch.tensor([pages - 1], dtype=torch.int32, device="cuda"),
                     torch.tensor([pages - 3], dtype=torch.int32, device="cuda"))
    assert torch.equal(pool[0, pages - 3], pool[0, pages - 1])
    assert not pool[0, :8].any()
    cache.raise_on_error()
