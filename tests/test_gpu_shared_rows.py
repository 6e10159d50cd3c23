"""Attention behind shared prefixes where cu_tokens is out of range or descends, at
the edges of groups as well as inside: the sequences that it says nothing wrong of
are right, as in attention that shares nothing, whatever an earlier call has left
in the workspace."""
import numpy as np
import pytest

from cache_common import attend_bound, attend_exact
from gpu_common import torch_mod
from test_gpu_attend_shared import Groups

pytestmark = pytest.mark.gpu

MORE = 8   # tokens that a sequence may have beyond its own when an entry dips

# sequences, groups ([first, end), shared slots), heads of a group, kv_heads, head_dim, page, type, most tokens, own slots
BATCHES = {
    "few": (6, [(0, 3, 64), (3, 6, 100)], 2, 2, 64, 16, "bf16", 3, [5, 0, 40, 17, 33, 9]),
    "few_long": (6, [(0, 3, 64), (3, 6, 100)], 2, 2, 128, 32, "f16", 3, [5, 1100, 40, 1030, 1200, 9]),
    "many": (100, [(0, 40, 130), (40, 41, 300), (41, 93, 97)], 4, 2, 64, 16, "f16", 3, None),
    "many_long": (100, [(0, 40, 130), (40, 60, 97), (60, 100, 64)], 16, 2, 128, 32, "bf16", 6, None),
}
# where an entry is changed: the first, one inside a group, the edge between two groups, the last one
PLACES = {"few": (0, 2, 3, 6), "few_long": (0, 2, 3, 6), "many": (0, 20, 41, 93, 100), "many_long": (0, 20, 40, 60, 100)}


def build(tcd, name, room):
    batch, groups, group, hkv, d, page, dt, most, own = BATCHES[name]
    rng = np.random.default_rng(17)
    tokens = rng.integers(1, most + 1, batch)
    own = rng.integers(0, 90, batch) if own is None else np.array(own)
    for lo, hi, shared in groups:
        own[lo:hi] += shared
    w = Groups(tcd, [int(x) + MORE for x in tokens], [int(x) for x in own], groups, dt, hkv, d, page, 5, room, group)
    w.real = tokens
    w.cu_real = np.concatenate(([0], np.cumsum(tokens))).astype(np.int64)
    return w, group * hkv


def change(cu, place, kind, n):
    cu = cu.copy()
    if kind == "past":
        cu[place] = n + 77
    elif kind == "negative":
        cu[place] = -3
    else:
        cu[place] = cu[1] + 2 if place == 0 else max(0, cu[place] - 5)
    return cu


def spans(cu, n):
    """Rows of each sequence, or None."""
    return [(int(a), int(b)) if 0 <= a <= b <= n else None for a, b in zip(cu, cu[1:])]


def check(w, kv, q64, out, lse, cu, bounds):
    """Every sequence that is in order is right; elements of a row that several of them have are any one's."""
    n, hq, d = q64.shape
    at = spans(cu, n)
    assert w.status.tolist() == [0 if s else bounds for s in at]
    got, sums = out.double().cpu().numpy(), lse.double().cpu().numpy()
    fits, sums_fit, owned = np.zeros((n, hq, d), bool), np.zeros((n, hq), bool), np.zeros(n, bool)
    group = hq // w.kv_heads
    for b, s in enumerate(at):
        if not s or s[0] == s[1]:
            continue
        rows, c = np.arange(*s), w.ctx_list[b]
        total = c + len(rows)
        seen = np.arange(total)[None] <= c + np.arange(len(rows))[:, None]
        part = kv[b][:, :, :total]
        want, mag, ls, big = attend_exact(q64[rows], part, seen, d ** -0.5, group)
        vsum = np.einsum("tn,hnd->thd", seen.astype(np.float64), np.abs(part[1])).repeat(group, axis=1)
        fits[rows] |= np.abs(got[rows] - want) <= attend_bound(w.dt, want, mag, big, vsum, d)
        sums_fit[rows] |= np.abs(sums[rows] - ls) <= 2 * (d + 4) * 2.0 ** -24 * big + 2.0 ** -20 * (1 + np.abs(ls))
        owned[rows] = True
    fits = fits.all(axis=(1, 2)) & sums_fit.all(axis=1)
    assert fits[owned].all(), np.argwhere(owned & ~fits)[:8].ravel().tolist()
    return owned


@pytest.mark.parametrize("room", [17, 0])
@pytest.mark.parametrize("kind", ["past", "negative", "descent"])
@pytest.mark.parametrize("name", list(BATCHES))
def test_entries_out_of_order(tcd, name, kind, room):
    torch = torch_mod()
    w, hq = build(tcd, name, room)
    n = int(w.cu_real[-1])
    for place in PLACES[name]:
        w.cu.copy_(torch.from_numpy(w.cu_real))
        w.fill()                                     # (another request's numbers are left in the workspace)
        q, _ = w.normal(n, hq, w.head_dim)
        w.attend(q, lse=True)
        assert not w.status.any()
        kv = w.fill()
        q, q64 = w.normal(n, hq, w.head_dim)
        cu = change(w.cu_real, place, kind, n)
        w.cu.copy_(torch.from_numpy(cu))
        out, lse = w.attend(q, lse=True)
        check(w, kv, q64, out, lse, cu, tcd.TC_ERR_BOUNDS)


@pytest.mark.parametrize("name", ["few", "many"])
def test_rows_of_no_sequence_are_left_behind_a_dip(tcd, name):
    """The rows of sequences that the entries leave out stay as they were, as in attention that shares nothing."""
    torch = torch_mod()
    w, hq = build(tcd, name, 17)
    n, kv = int(w.cu_real[-1]), w.fill()
    q, q64 = w.normal(n, hq, w.head_dim)
    w.cu.copy_(torch.from_numpy(w.cu_real))
    w.attend(q)
    cu = change(w.cu_real, PLACES[name][1], "past", n)
    w.cu.copy_(torch.from_numpy(cu))
    out, lse = w.attend(q, lse=True)
    owned = torch.from_numpy(check(w, kv, q64, out, lse, cu, tcd.TC_ERR_BOUNDS)).cuda()
    assert not bool(owned.all()) and bool((out[~owned] == 55).all()) and bool((lse[~owned] == 55).all())


@pytest.mark.parametrize("name", ["few", "many_long"])
def test_in_a_graph(tcd, name):
    """The entries are read when the graph runs: out of order, in order again, and gathered errors."""
    torch = torch_mod()
    w, hq = build(tcd, name, 17)
    n, kv = int(w.cu_real[-1]), w.fill()
    q, q64 = w.normal(n, hq, w.head_dim)
    w.cu.copy_(torch.from_numpy(w.cu_real))
    want, lse = w.attend(q, lse=True)
    check(w, kv, q64, want, lse, w.cu_real, 0)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out, lse = w.attend(q, lse=True)
    for place in PLACES[name]:
        cu = change(w.cu_real, place, "past", n)
        w.cu.copy_(torch.from_numpy(cu))
        out.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        check(w, kv, q64, out, lse, cu, tcd.TC_ERR_BOUNDS)
        w.cu.copy_(torch.from_numpy(w.cu_real))
        g.replay()
        torch.cuda.synchronize()
        assert not w.status.any() and torch.equal(out, want)
