"""Attention where the work of a call is cut: items of odd groups over many
workers, and many short items in one worker (GPU).  Rows at the places where
tiles, items and parts meet are compared with the definition in 64 bits; the
bounds are those of the other attention tests."""
import numpy as np
import pytest

from cache_common import Batch, attend_bound, attend_exact, compare
from gpu_common import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tcd():
    from trie_constrained_decoding_gb300 import binding
    return binding


CASES = [
    # tokens, ctx, q_heads, kv_heads, head_dim, page, type
    ([1700, 3, 0, 900], [1000, 2000, 5, 0], 14, 2, 128, 32, "bf16"),   # 18 tokens a tile
    ([1500, 700, 1], [0, 2999, 4097], 24, 8, 64, 16, "f16"),           # 42
    ([2501], [0], 10, 2, 128, 64, "bf16"),                             # 25
    ([130, 1], [6000, 9000], 100, 1, 64, 128, "bf16"),                 # 1
    ([1] * 200, [20 + 3 * (i % 21) for i in range(200)], 8, 8, 128, 64, "bf16"),
    ([1 + i % 3 for i in range(220)], [(37 * i) % 90 for i in range(220)], 12, 4, 64, 16, "f16"),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_cut_work(tcd, case):
    torch = torch_mod()
    tokens, ctx, hq, hkv, d, page, dt = CASES[case]
    w = Batch(tcd, tokens, ctx, dt, hkv, d, page, seed=300 + case)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, d)
    out = torch.full(q.shape, 55.0, dtype=q.dtype, device="cuda")
    lse = torch.full((w.n, hq), 55.0, device="cuda")
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, max(tokens), lse=lse, status=w.status)
    torch.cuda.synchronize()
    assert w.status.cpu().tolist() == [0] * len(tokens)
    got, sums = out.double().cpu().numpy().reshape(q64.shape), lse.double().cpu().numpy()
    assert np.isfinite(got).all() and not (got == 55.0).all(axis=(1, 2)).any()
    group = hq // hkv
    step = 2 * (128 // group)
    for b, (t, c) in enumerate(zip(tokens, ctx)):
        rows = sorted({r for r in (0, 1, step // 2 - 1, step // 2, step - 1, step, 7 * step, t // 2, t - 2, t - 1)
                       if 0 <= r < t})
        if not rows or (len(tokens) > 50 and b % 9):
            continue
        lo = w.cu_host[b]
        at = lo + np.array(rows)
        seen = np.arange(t + c)[None, :] <= c + np.array(rows)[:, None]
        want, mag, ls, big = attend_exact(q64[at], kv[b], seen, d ** -0.5, group)
        vsum = np.einsum("tn,hnd->thd", seen.astype(np.float64), np.abs(kv[b][1])).repeat(group, axis=1)
        compare(f"sequence {b}", got[at], want, attend_bound(dt, want, mag, big, vsum, d))
        compare(f"lse {b}", sums[at], ls, 2 * (d + 4) * 2.0 ** -24 * big + 2.0 ** -20 * (1 + np.abs(ls)))
    # the cuts depend on the lengths only: the same bits again
    again = torch.zeros_like(out)
    w.cache.attend(0, q, w.cu, w.ctx, w.table, again, max(tokens), status=w.status)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
