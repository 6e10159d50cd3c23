"""Attention of sequences that share a prefix, against its definition in 64 bits:
groups of different sizes, prefixes that end inside a page or a tile, drafts,
prompts and single tokens, sequences without tokens or without a group; errors,
streams, graphs and workspaces."""
import numpy as np
import pytest

from cache_common import Batch, ancestors, attend_bound, attend_exact, compare, mask_words, random_parents
from gpu_common import torch_mod

pytestmark = pytest.mark.gpu


class Groups(Batch):
    """A batch whose groups ([first, end) sequences, shared slots) hold their whole shared pages in common.

    room: MB of slots that the page tables have place for, and 4 for each row that a sequence has in the mean, of up to
    `heads` heads of a group (up to 16 and 4 contexts are read sequence by sequence)."""

    def __init__(self, tcd, tokens, ctx, groups, dt="bf16", kv_heads=2, head_dim=128, page=16, seed=0, room=17, heads=16):
        place = (room << 20) + (4 << 20) * heads * sum(tokens) // len(tokens)
        wide = place // (len(tokens) * page * kv_heads * head_dim * 4) + 1 if room else 2
        super().__init__(tcd, tokens, ctx, dt, kv_heads, head_dim, page, seed=seed, extra_width=wide)
        torch = torch_mod()
        self.groups = groups
        self.prefix = [0] * len(tokens)
        self.leader = list(range(len(tokens)))
        for lo, hi, shared in groups:
            for b in range(lo, hi):
                self.prefix[b] = shared // page * page
                self.leader[b] = lo
                self.table_host[b, :shared // page] = self.table_host[lo, :shared // page]
        self.table = torch.from_numpy(self.table_host).cuda()
        edges = [groups[0][0]] + [hi for _, hi, _ in groups]
        assert all(g[0] == e for g, e in zip(groups, edges))
        self.cu_seqs = torch.tensor(edges, dtype=torch.int32, device="cuda")
        self.shared = torch.tensor([g[2] for g in groups], dtype=torch.int32, device="cuda")

    def fill(self):
        torch = torch_mod()
        got = []
        for b, (t, c) in enumerate(zip(self.tokens, self.ctx_list)):
            lo = self.prefix[b] if self.leader[b] != b else 0
            dev, host = self.normal(2, self.kv_heads, t + c - lo, self.head_dim)
            if lo:
                host = np.concatenate((got[self.leader[b]][:, :, :lo], host), 2)
            pages, offs = self.slots(b, lo, t + c)
            if t + c > lo:
                self.pool[0, torch.from_numpy(pages).long().cuda(), :, :, torch.from_numpy(offs).cuda()] = \
                    dev.permute(2, 0, 1, 3)
            got.append(host)
        return got

    def attend(self, q, masks=None, words=1, lse=False, scale=None, out=None, **kw):
        torch = torch_mod()
        out = torch.full(q.shape, 55.0, dtype=q.dtype, device="cuda") if out is None else out
        ls = torch.full(q.shape[:2], 55.0, device="cuda") if lse else None
        kw.setdefault("status", self.status)
        self.cache.attend_shared(0, q, self.cu, self.ctx, self.table, out, kw.pop("max_tokens", max(self.tokens)),
                                 self.cu_seqs, self.shared, scale=scale,
                                 tree=None if masks is None else mask_words(masks, words), lse=ls, **kw)
        return out, ls

    def check(self, kv, q64, out, masks=None, lse=None, scale=None, rows=None, skip=()):
        hq, d = q64.shape[1], self.head_dim
        scale = d ** -0.5 if scale is None else scale
        seen, got = self.seen(masks), out.double().cpu().numpy()
        assert [c for b, c in enumerate(self.status.cpu().tolist()) if b not in skip] == \
            [0] * (len(self.tokens) - len(skip))
        group = hq // self.kv_heads
        for b, t in enumerate(self.tokens):
            use = np.array([r for r in (range(t) if rows is None else rows) if r < t], dtype=int)
            if b in skip or not len(use):
                continue
            at = self.cu_host[b] + use
            want, mag, ls, big = attend_exact(q64[at], kv[b], seen[b][use], scale, group)
            vsum = np.einsum("tn,hnd->thd", seen[b][use].astype(np.float64), np.abs(kv[b][1])).repeat(group, axis=1)
            compare(f"sequence {b}", got[at], want, attend_bound(self.dt, want, mag, big, vsum, d))
            if lse is not None:
                empty = np.isneginf(ls)
                g = lse.double().cpu().numpy()[at]
                assert np.array_equal(np.isneginf(g), empty)
                tol = 2 * (d + 4) * 2.0 ** -24 * big + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, ls)))
                compare(f"lse {b}", np.where(empty, 0, g), np.where(empty, 0, ls), tol)


CASES = [
    # tokens, slots behind the shared ones, groups, q_heads, kv_heads, head_dim, page, type
    ([1, 1], [0, 0], [(0, 2, 16)], 1, 1, 128, 16, "bf16"),
    ([1, 1, 1, 1], [3, 0, 21, 130], [(0, 4, 37)], 8, 2, 64, 16, "bf16"),
    ([1] * 5, [1, 2, 3, 4, 200], [(0, 5, 640)], 4, 4, 128, 64, "f16"),
    ([2, 0, 7, 1, 3], [0, 5, 120, 0, 9], [(0, 5, 300)], 8, 2, 128, 32, "f16"),
    ([1] * 40, list(range(0, 400, 10)), [(0, 40, 1000)], 32, 8, 64, 128, "bf16"),
    ([1, 2, 3, 4, 5, 6], [9, 8, 7, 6, 5, 4], [(0, 2, 129), (2, 3, 500), (3, 6, 64)], 12, 4, 64, 16, "bf16"),
    ([3] * 7, [11] * 7, [(1, 3, 200), (3, 3, 70), (3, 6, 260)], 28, 4, 128, 32, "f16"),
    ([1] * 3, [5, 600, 30], [(0, 3, 0)], 4, 2, 128, 16, "bf16"),
    ([1] * 3, [5, 600, 30], [(0, 3, 15)], 4, 2, 64, 16, "f16"),
    ([64, 65, 31, 32], [64, 63, 1, 96], [(0, 4, 513)], 8, 1, 128, 64, "bf16"),
    ([260, 13], [13, 700], [(0, 2, 333)], 4, 2, 64, 16, "f16"),
    ([300, 7, 150], [0, 0, 0], [(0, 3, 2048)], 16, 2, 128, 32, "bf16"),
    ([1] * 130, [7] * 130, [(0, 65, 256), (65, 130, 2000)], 3, 1, 64, 128, "bf16"),
    ([3, 2], [70, 1], [(0, 2, 48)], 128, 1, 64, 16, "bf16"),
    ([2, 3], [9, 0], [(0, 2, 129)], 100, 1, 128, 16, "f16"),
    # rests that are just short enough for a kernel of their own, and just too long or with too many rows
    ([1, 1, 1, 1], [1023, 1024, 1022, 0], [(0, 4, 64)], 2, 1, 64, 32, "bf16"),
    ([16, 17, 15, 1], [60, 60, 1009, 1023], [(0, 4, 64)], 8, 2, 128, 64, "bf16"),
    ([4, 3, 1, 2], [63, 64, 65, 129], [(0, 4, 128)], 4, 1, 128, 64, "f16"),
    ([8, 5, 1, 7], [64, 59, 127, 1], [(0, 4, 128)], 4, 1, 64, 16, "f16"),
    ([16, 11, 1, 13], [48, 500, 63, 0], [(0, 4, 96)], 4, 1, 128, 32, "bf16"),
    ([64, 64], [0, 960], [(0, 2, 16)], 3, 3, 64, 16, "bf16"),
]


def build(tcd, case, seed, room=17):
    tokens, behind, groups, hq, hkv, d, page, dt = case
    ctx = list(behind)
    for lo, hi, shared in groups:
        for b in range(lo, hi):
            ctx[b] += shared
    return Groups(tcd, tokens, ctx, groups, dt, hkv, d, page, seed, room, hq // hkv), hq


@pytest.mark.parametrize("room", [17, 0])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_causal(tcd, case, room):
    w, hq = build(tcd, CASES[case], case, room)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, w.head_dim)
    out, lse = w.attend(q, lse=True)
    w.check(kv, q64, out, lse=lse, rows=list(range(5)) + list(range(5, 400, 37)))


@pytest.mark.parametrize("case", [i for i, c in enumerate(CASES) if max(c[0]) <= 64])
@pytest.mark.parametrize("room", [17, 0])
def test_drafts(tcd, case, room):
    w, hq = build(tcd, CASES[case], 50 + case, room)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, w.head_dim)
    masks = [m for n in w.tokens for m in ancestors(random_parents(w.rng, n))]
    out, lse = w.attend(q, masks, lse=True)
    w.check(kv, q64, out, masks, lse=lse)


# One prefix in many parts: sequences, heads of a group, kv_heads, head_dim, page, type, prefix.  A row's parts are added
# up by one thread or by two, as the call's tokens and heads fill tasks: few rows, rows that end inside a task, and on
# either side of the change (9 and 10 tiles of 64 tokens with 152 SMs).
LONG = [
    (2, 1, 1, 128, 64, "bf16", 20011), (2, 1, 1, 64, 16, "f16", 3001), (9, 4, 8, 128, 64, "bf16", 3011),
    (75, 3, 3, 64, 32, "f16", 2500), (64, 4, 8, 128, 64, "f16", 1500), (64, 4, 9, 128, 64, "bf16", 1300),
    (64, 4, 10, 128, 64, "bf16", 1300), (70, 4, 8, 64, 128, "bf16", 1500), (3, 100, 2, 128, 32, "bf16", 2100),
]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_long_prefix(tcd, case):
    batch, group, hkv, d, page, dt, prefix = LONG[case]
    tokens = [1 + b % 2 for b in range(batch)] if batch < 64 else [1] * batch
    w = Groups(tcd, tokens, [prefix + 7 * b % 90 for b in range(batch)], [(0, batch, prefix)], dt, hkv, d, page, 90 + case,
               heads=group)
    kv = w.fill()
    q, q64 = w.normal(w.n, group * hkv, d)
    out, lse = w.attend(q, lse=True)
    w.check(kv, q64, out, lse=lse)
    again, lse2 = w.attend(q, lse=True)
    assert torch_mod().equal(out, again) and torch_mod().equal(lse, lse2)


# Many sequences at once (more items than the GPU has SMs): heads of a group, kv_heads, head_dim, page, type, most tokens
MANY = [
    (4, 2, 128, 64, "bf16", 1), (4, 2, 128, 16, "f16", 16), (1, 2, 64, 128, "bf16", 64), (7, 2, 64, 32, "f16", 9),
    (16, 2, 128, 128, "bf16", 4), (3, 2, 64, 16, "bf16", 21), (64, 2, 128, 32, "f16", 1), (2, 2, 128, 64, "bf16", 40),
    (70, 2, 64, 64, "bf16", 2),
]


def many(tcd, case, seed):
    """100 sequences in three groups (the last seven in none): no token to more than a short rest may have, nothing of
    their own to more slots than that."""
    group, hkv, d, page, dt, most = MANY[case]
    rng = np.random.default_rng(seed)
    tokens = rng.integers(0, most + 1, 100)
    tokens[:8] = [1, most, 0, 1, most, 1, 1, max(1, 64 // group)]
    behind = rng.integers(0, 260, 100)
    behind[:8] = [0, 64 - min(most, 64), 5, 63, 64, 1024, 1023, 700]
    groups = [(0, 40, 130), (40, 41, 300), (41, 93, 3 * page + 1)]
    ctx = behind + np.repeat([g[2] for g in groups] + [0], [40, 1, 52, 7])
    return Groups(tcd, [int(x) for x in tokens], [int(x) for x in ctx], groups, dt, hkv, d, page, seed,
                  heads=group), group * hkv


@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_sequences(tcd, case, drafts):
    w, hq = many(tcd, case, 60 + case)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, w.head_dim)
    words = -(-max(w.tokens) // 64)
    masks = [m for n in w.tokens for m in ancestors(random_parents(w.rng, n))] if drafts else None
    out, lse = w.attend(q, masks, words, lse=True)
    w.check(kv, q64, out, masks, lse=lse, rows=[0, 1, 2, 7, 15, 20, 39, 63])


def test_many_sequences_with_values_that_are_not_finite(tcd):
    """Infinities and NaN in drafted values of many sequences: to the rows that see them, and to no other."""
    torch = torch_mod()
    for case in (1, 7):
        w, hq = many(tcd, case, 3)
        w.fill()
        q, _ = w.normal(w.n, hq, w.head_dim)
        masks = [m for n in w.tokens for m in ancestors(random_parents(w.rng, n))]
        want = w.attend(q, masks)[0].clone()
        plus, nan = torch.zeros_like(want, dtype=torch.bool), torch.zeros_like(want, dtype=torch.bool)
        group = hq // w.kv_heads
        for b, n in enumerate(w.tokens):
            if n < 2 or b % 3:
                continue
            for x, column, value, to in ((n - 1, 5, float("inf"), plus), (n // 2, 9, float("nan"), nan)):
                page, off = w.slots(b, w.ctx_list[b] + x, w.ctx_list[b] + x + 1)
                w.pool[0, int(page[0]), 1, 1, int(off[0]), column] = value
                for i in range(n):
                    if masks[w.cu_host[b] + i] >> x & 1:
                        to[w.cu_host[b] + i, group:, column] = True
        out = w.attend(q, masks)[0]
        keep = ~(plus | nan)
        assert torch.equal(out[keep], want[keep])
        assert bool((out[plus] == float("inf")).all()) and bool(out[nan].isnan().all())


def test_many_sequences_in_graphs_and_out_of_them(tcd):
    """The same bits each time, in a graph that is replayed beside plain calls on another stream."""
    torch = torch_mod()
    w, hq = many(tcd, 1, 5)
    w.fill()
    q, _ = w.normal(w.n, hq, w.head_dim)
    want = w.attend(q)[0].clone()
    for _ in range(3):
        assert torch.equal(w.attend(q)[0], want)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = torch.zeros_like(want), torch.zeros_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w.attend(q, out=a, status=None)
    for _ in range(20):
        with torch.cuda.stream(s):
            g.replay()
        w.attend(q, out=b, status=None, stream=t)
    w.cache.raise_on_error()
    assert torch.equal(a, want) and torch.equal(b, want)


def test_many_sequences_with_errors(tcd):
    """Errors of single sequences among many; a wait that runs out; and the next call is right."""
    torch = torch_mod()
    w, hq = many(tcd, 0, 6)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, w.head_dim)
    good = w.attend(q)[0].clone()
    w.check(kv, q64, good)
    w.ctx[3] = 10                                   # its group shares 128
    w.table[4, 0] = w.table[6, 4]                   # a valid page, but another one
    w.table[9, -1] = -5                             # (not read)
    w.table[5, 2] = 1 << 20                         # a page that does not exist, behind the prefix
    out, _ = w.attend(q)
    assert [i for i, c in enumerate(w.status.tolist()) if c] == [3, 4, 5]
    w.check(kv, q64, out, skip=(3, 4, 5))
    w, hq = many(tcd, 0, 6)
    w.fill()
    w.cache.attend_wait_test(True, 2000)
    w.attend(q)
    assert tcd.TC_ERR_DEVICE_TIMEOUT in w.status.tolist()
    w.cache.attend_wait_test(False, 0)
    kv = w.fill()
    out, _ = w.attend(q)
    assert w.status.tolist() == [0] * 100
    w.check(kv, q64, out)


def test_pages_far_into_a_large_pool(tcd):
    """Offsets in the cache beyond 2^32 bytes."""
    torch = torch_mod()
    w, hq = many(tcd, 4, 8)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, w.head_dim)
    want = w.attend(q)[0].clone()
    w.check(kv, q64, want, rows=[0, 1, 3])
    pages = 36000 + w.pages
    pool = torch.empty((1, pages) + tuple(w.pool.shape[2:]), dtype=w.pool.dtype, device="cuda")
    assert pool.numel() > 1 << 31
    pool[:, -w.pages:] = w.pool
    w.table += 36000
    cache = tcd.KvCache(pool)
    out = torch.empty_like(q)
    cache.attend_shared(0, q, w.cu, w.ctx, w.table, out, max(w.tokens), w.cu_seqs, w.shared, status=w.status)
    assert w.status.tolist() == [0] * 100 and torch.equal(out, want)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_many_sequences_scales(tcd, scale):
    w, hq = many(tcd, 3, 7)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, w.head_dim)
    out, lse = w.attend(q, lse=True, scale=scale)
    w.check(kv, q64, out, lse=lse, scale=scale, rows=[0, 3, 8])


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(tcd, scale):
    w, hq = build(tcd, CASES[3], 7)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, w.head_dim)
    out, lse = w.attend(q, lse=True, scale=scale)
    w.check(kv, q64, out, lse=lse, scale=scale)


def test_rows_that_see_nothing(tcd):
    """Empty masks: with a prefix the row sees that only; without one it is zero.  The last group shares nothing."""
    w = Groups(tcd, [2, 1, 2, 2], [32, 32, 0, 0], [(0, 2, 32), (2, 4, 0)], seed=3)
    kv = w.fill()
    q, q64 = w.normal(w.n, 4, 128)
    masks = [0, 1, 0, 0, 2, 1, 0]
    out, lse = w.attend(q, masks, lse=True)
    w.check(kv, q64, out, masks, lse=lse)
    assert bool((out[3] == 0).all()) and bool((out[6] == 0).all())


def test_far_prefix_and_near_rest(tcd):
    """Maxima of the two parts far apart, either way: one of them weighs nothing, and nothing overflows."""
    torch = torch_mod()
    for dt in ("bf16", "f16"):
        w = Groups(tcd, [1, 1], [64, 96], [(0, 2, 64)], dt, 1, 64, 16, seed=1)
        kv = w.fill()
        q, _ = w.normal(2, 2, 64)
        big = torch.full((64,), 8.0, dtype=q.dtype, device="cuda")
        q[:] = big
        for at, where in ((0, (0, 3)), (1, (1, 70))):      # a key of the prefix, then one of a sequence's own
            page, off = w.slots(*[where[0], where[1], where[1] + 1])
            w.pool[0, int(page[0]), 0, 0, int(off[0])] = big
            kv[where[0]][0, 0, where[1]] = 8.0
            if at == 0:
                kv[1][0, 0, 3] = 8.0
            out, lse = w.attend(q, lse=True)
            w.check(kv, q.double().cpu().numpy(), out, lse=lse)


def test_equals_attend(tcd):
    """The same call without sharing: within two roundings of the weights and the output."""
    w, hq = build(tcd, CASES[4], 9)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, w.head_dim)
    out, _ = w.attend(q)
    plain = out.clone()
    w.cache.attend(0, q, w.cu, w.ctx, w.table, plain, 1, status=w.status)
    w.check(kv, q64, plain)
    w.check(kv, q64, out)


def test_garbage_beside_the_slots_seen(tcd):
    """NaN and infinities among drafted values of other branches, and behind the end, change nothing."""
    torch = torch_mod()
    w = Groups(tcd, [4, 3], [40, 33], [(0, 2, 32)], seed=4)
    kv = w.fill()
    q, q64 = w.normal(w.n, 4, 128)
    masks = [1, 2, 5, 8, 1, 2, 4]
    want = w.attend(q, masks)[0].clone()
    w.check(kv, q64, want, masks)
    page, off = w.slots(0, 41, 42)                # draft 1 of sequence 0: its own row alone sees it
    w.pool[0, int(page[0]), 1, :, int(off[0])] = float("nan")
    out = w.attend(q, masks)[0]
    keep = [0, 2, 3, 4, 5, 6]
    assert torch.equal(out[keep], want[keep]) and bool(out[1].isnan().all())


@pytest.mark.parametrize("hq", [1, 6, 15])
def test_infinite_values(tcd, hq):
    """An infinity among the drafted values reaches the rows that see it, unchanged, and no other row; and so does one
    behind it that another part of the rows' slots holds."""
    torch = torch_mod()
    for dt, d in (("bf16", 64), ("f16", 128)):
        w = Groups(tcd, [4, 3], [150, 33], [(0, 2, 32)], dt, 1, d, seed=4)
        w.fill()
        q, _ = w.normal(w.n, hq, d)
        masks = [1, 2, 5, 8, 1, 2, 4]
        want = w.attend(q, masks)[0].clone()
        page, off = w.slots(0, 152, 153)              # draft 2 of sequence 0: its own row alone sees it
        w.pool[0, int(page[0]), 1, 0, int(off[0]), 3] = float("inf")
        w.pool[0, int(page[0]), 1, 0, int(off[0]), 5] = float("-inf")
        out = w.attend(q, masks)[0]
        inf = torch.zeros_like(out, dtype=torch.bool)
        inf[2, :, 3], inf[2, :, 5] = True, True
        assert torch.equal(out[~inf], want[~inf])
        assert bool((out[2, :, 3] == float("inf")).all()) and bool((out[2, :, 5] == -float("inf")).all())


def test_rows_of_no_sequence_are_left(tcd):
    torch = torch_mod()
    w, hq = build(tcd, CASES[5], 2)
    kv = w.fill()
    q, q64 = w.normal(w.n + 6, hq, w.head_dim)
    w.cu_host = w.cu_host + 2
    w.cu = torch.from_numpy(w.cu_host).cuda()
    out, lse = w.attend(q, lse=True)
    w.check(kv, q64, out, lse=lse)
    for x in (out, lse):
        assert bool((x[:2] == 55).all()) and bool((x[w.n + 2:] == 55).all())


def test_slices_of_wider_rows(tcd):
    torch = torch_mod()
    w, hq = build(tcd, CASES[1], 2)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, w.head_dim)
    wide = torch.full((w.n, (hq + 3) * w.head_dim + 8), 55.0, dtype=q.dtype, device="cuda")
    wide[:, 8:8 + hq * w.head_dim] = q.flatten(1)
    got = torch.full_like(wide, 55.0)
    w.attend(wide[:, 8:8 + hq * w.head_dim].unflatten(1, (hq, -1)),
             out=got[:, 8:8 + hq * w.head_dim].unflatten(1, (hq, -1)))
    w.check(kv, q64, got[:, 8:8 + hq * w.head_dim].unflatten(1, (hq, -1)))
    got[:, 8:8 + hq * w.head_dim] = 55
    assert bool((got == 55).all())


@pytest.mark.parametrize("room", [17, 0])
def test_errors_by_sequence(tcd, room):
    """A page that differs, fewer slots than shared: that sequence; a length out of range: its group."""
    torch = torch_mod()
    case = ([1] * 6, [5] * 6, [(0, 3, 64), (3, 6, 100)], 4, 2, 64, 16, "bf16")
    bounds = tcd.TC_ERR_BOUNDS

    def fresh():
        w, hq = build(tcd, case, 1, room)
        kv = w.fill()
        q, q64 = w.normal(w.n, hq, 64)
        return w, kv, q, q64

    w, kv, q, q64 = fresh()
    w.table[1, 2] = w.table[3, 0]                   # a valid page, but another one
    out, _ = w.attend(q)
    assert w.status.tolist() == [0, bounds, 0, 0, 0, 0]
    w.check(kv, q64, out, skip=(1,))
    w, kv, q, q64 = fresh()
    w.ctx[4] = 40                                   # its group shares 96
    out, _ = w.attend(q)
    assert w.status.tolist() == [0, 0, 0, 0, bounds, 0]
    w.check(kv, q64, out, skip=(4,))
    for bad in (-1, 1 << 30):
        w, kv, q, q64 = fresh()
        w.shared[0] = bad
        out, _ = w.attend(q)
        assert w.status.tolist() == [bounds] * 3 + [0] * 3
        w.check(kv, q64, out, skip=(0, 1, 2))
    for edges in ([0, 4, 3], [-1, 3, 6], [0, 3, 7], [3, 0, 6]):
        w, kv, q, q64 = fresh()
        w.cu_seqs.copy_(torch.tensor(edges))
        out, _ = w.attend(q)
        assert w.status.tolist() == [bounds] * 6
        assert bool((out == 55).all())
    w, kv, q, q64 = fresh()
    w.cu[2] = 77                                    # rows out of range: sequences 1 and 2
    w.attend(q)
    assert w.status.tolist()[1:3] == [bounds] * 2 and w.status.tolist()[3:] == [0] * 3
    w, kv, q, q64 = fresh()
    out, _ = w.attend(q, max_tokens=0)
    assert w.status.tolist() == [bounds] * 6
    # errors without a status are gathered
    w.attend(q, max_tokens=0, status=None)
    w.attend(q, status=None)
    with pytest.raises(tcd.TcError):
        w.cache.raise_on_error()
    w.cache.raise_on_error()


def test_refusals(tcd):
    torch = torch_mod()
    w, hq = build(tcd, CASES[1], 2)
    w.fill()
    q, _ = w.normal(w.n, hq, w.head_dim)
    need = w.cache.shared_workspace_bytes(w.n, hq)
    assert need > w.cache.workspace_bytes
    with pytest.raises(tcd.TcError):
        w.attend(q, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    good = w.attend(q)[0].clone()
    assert torch.equal(w.attend(q, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))[0], good)
    shared, edges = w.shared, w.cu_seqs
    for s, e, kind in ((shared.long(), edges, ValueError), (shared, edges[:1], ValueError),
                       (shared[:0], edges[:1], tcd.TcError), (shared.cpu(), edges, ValueError),
                       (shared.new_zeros(5), edges.new_zeros(6), tcd.TcError)):
        w.shared, w.cu_seqs = s, e
        with pytest.raises(kind):
            w.attend(q)


def test_no_tokens(tcd):
    torch = torch_mod()
    w = Groups(tcd, [0, 0], [20, 30], [(0, 2, 16)], seed=1)
    w.fill()
    q = torch.zeros((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    w.attend(q, max_tokens=0)
    assert w.status.tolist() == [0, 0]


def test_wait_that_runs_out(tcd):
    torch = torch_mod()
    w, hq = build(tcd, CASES[4], 2)
    w.fill()
    q, _ = w.normal(w.n, hq, w.head_dim)
    good = w.attend(q)[0].clone()
    w.cache.attend_wait_test(True, 2000)
    w.attend(q)
    assert w.status.tolist() == [tcd.TC_ERR_DEVICE_TIMEOUT] * len(w.tokens)
    w.cache.attend_wait_test(False, 0)
    assert torch.equal(w.attend(q)[0], good)
    assert w.status.tolist() == [0] * len(w.tokens)


def test_workspaces_grow_with_calls_and_graphs(tcd):
    """Calls of more and more tokens on one object, in one graph, in graphs side by side and beside plain calls."""
    torch = torch_mod()
    # one cache object for all, over the largest batch's pool
    big, hq = build(tcd, ([1] * 60, [9] * 60, [(0, 60, 512)], 8, 2, 128, 64, "bf16"), 5)
    big.fill()
    q, _ = big.normal(60, hq, 128)

    def call(n, out, stream=None):
        """The first n sequences."""
        big.cache.attend_shared(0, q[:n], big.cu[:n + 1], big.ctx[:n], big.table[:n], out, 1, edges[n], big.shared,
                                stream=stream)

    sizes = (2, 17, 60)
    edges = {n: torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in sizes}
    want = {}
    for n in sizes:
        want[n] = torch.empty_like(q[:n])
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


def test_same_bits_each_time(tcd):
    torch = torch_mod()
    w, hq = build(tcd, CASES[12], 2)
    w.fill()
    q, _ = w.normal(w.n, hq, w.head_dim)
    first = w.attend(q)[0].clone()
    for _ in range(5):
        assert torch.equal(w.attend(q)[0], first)


def test_forked_pages(tcd):
    """The pages that a pool hands out: a prompt is forked, the last, partly filled page is copied on its first write."""
    torch = torch_mod()
    page, prompt, n = 16, 37, 3
    pool = tcd.PagePool(32, page)
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = tcd.KvCache(torch.randn((1, 32, 2, 2, page, 64), generator=g, device="cuda").bfloat16())
    seqs = [pool.open()]
    pool.reserve(seqs[0], 0, prompt)
    seqs += [pool.fork(seqs[0], prompt) for _ in range(n - 1)]
    for s in seqs:
        for a, b in pool.reserve(s, prompt, prompt + 1):
            cache.copy_pages(torch.tensor([a], dtype=torch.int32, device="cuda"),
                             torch.tensor([b], dtype=torch.int32, device="cuda"))
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, ctx, cu = ints(np.stack([pool.row(s, 700) for s in seqs])), ints([prompt] * n), ints(list(range(n + 1)))
    q = torch.randn((n, 8, 64), generator=g, device="cuda").bfloat16()
    out, plain = torch.empty_like(q), torch.empty_like(q)
    cache.attend_shared(0, q, cu, ctx, table, out, 1, ints([0, n]), ints([prompt]))
    cache.attend(0, q, cu, ctx, table, plain, 1)
    cache.raise_on_error()
    # two results of the same sums, in other orders: each within its weights' and its output's roundings
    v = cache.pool[0, :, 1].float().abs().max().item()
    assert float((out.float() - plain.float()).abs().max()) <= 4 * 2.0 ** -8 * v
