"""Waits that run out in the kernel for what sequences have for themselves behind a
shared prefix: every sequence that is reported as right is right, whatever an
earlier call has left in the workspace."""
import numpy as np
import pytest

from cache_common import attend_bound, attend_exact, compare
from gpu_common import torch_mod
from test_gpu_attend_shared import Groups

pytestmark = pytest.mark.gpu

KV_HEADS, D, PAGE = 4, 128, 16


def build(tcd, longs, group, short, long):
    """400 sequences in two groups: of the first 76 (as many items as the GPU has places for) none is long, of the others
    those that `longs` says.  Items are begun in order, so each place goes on to some of the others."""
    rng = np.random.default_rng(3)
    tokens = [long if b >= 76 and longs(b) else short for b in range(400)]
    own = rng.integers(3, 70, 400)
    w = Groups(tcd, tokens, [int(x) + s for x, s in zip(own, [48] * 200 + [80] * 200)], [(0, 200, 48), (200, 400, 80)],
               "bf16", KV_HEADS, D, PAGE, 11, heads=group)
    return w, group * KV_HEADS


def left_by_another_call(w, hq):
    """A workspace where every row's own part is there, of another call."""
    torch = torch_mod()
    need = w.cache.shared_workspace_bytes(w.n, hq)
    ws = torch.ones((need + 3) // 4, dtype=torch.float32, device="cuda")
    ws.view(torch.int32)[-(w.n * hq + 64):] = 1
    return ws


def check_right(w, kv, q64, out, status, every):
    got, hq, group = out.double().cpu().numpy(), q64.shape[1], q64.shape[1] // w.kv_heads
    for b in [b for b, c in enumerate(status) if c == 0][::every]:
        t, c = w.tokens[b], w.ctx_list[b]
        at = w.cu_host[b] + np.arange(t)
        seen = np.arange(t + c)[None] <= c + np.arange(t)[:, None]
        want, mag, _, big = attend_exact(q64[at], kv[b], seen, w.head_dim ** -0.5, group)
        vsum = np.einsum("tn,hnd->thd", seen.astype(np.float64), np.abs(kv[b][1])).repeat(group, axis=1)
        compare(f"sequence {b}", got[at], want, attend_bound(w.dt, want, mag, big, vsum, w.head_dim))


# heads of a group, tokens of short and long sequences, which are long
KINDS = [
    (16, 4, 5, lambda b: b % 16 != 5), (16, 4, 6, lambda b: b % 2 == 0), (4, 16, 17, lambda b: b % 8 != 5),
    (32, 1, 3, lambda b: b % 16 != 1), (16, 4, 5, lambda b: False),
]


@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_only_the_sequences_that_are_reported(tcd, kind):
    torch = torch_mod()
    group, short, long, longs = KINDS[kind]
    w, hq = build(tcd, longs, group, short, long)
    kv = w.fill()
    q, q64 = w.normal(w.n, hq, D)
    good = w.attend(q, workspace=left_by_another_call(w, hq))[0].clone()
    assert not w.status.any()
    check_right(w, kv, q64, good, w.status.tolist(), 9)
    for polls in (2000, 2300, 2600, 2900) * 3:
        w.cache.attend_wait_test(2, polls)
        out, _ = w.attend(q, workspace=left_by_another_call(w, hq))
        status = w.status.tolist()
        assert set(status) == {0, tcd.TC_ERR_DEVICE_TIMEOUT} and status[0] != 0
        # (the sums do not depend on who takes an item: the same bits)
        rows = torch.tensor([c == 0 for c in status], device="cuda").repeat_interleave(
            torch.tensor(w.tokens, device="cuda"))
        wrong = (out != good).flatten(1).any(1) & rows
        assert not bool(wrong.any()), np.unique(np.searchsorted(w.cu_host, wrong.nonzero()[:, 0].cpu().numpy(), "right") - 1)
    w.cache.attend_wait_test(False)
    assert torch.equal(w.attend(q)[0], good) and not w.status.any()


@pytest.mark.parametrize("group,n", [(16, 4), (64, 1), (2, 32), (32, 2)])
def test_an_item_that_one_warp_has_finished(tcd, group, n):
    """One of the two warps that have an item's rows gives up, the other one does not."""
    torch = torch_mod()
    w, hq = build(tcd, lambda b: False, group, n, n)
    w.fill()
    q, _ = w.normal(w.n, hq, D)
    good = w.attend(q)[0].clone()
    assert not w.status.any()
    for polls in (2000, 2500) * 3:
        w.cache.attend_wait_test(3, polls)
        out, _ = w.attend(q, workspace=left_by_another_call(w, hq))
        status = w.status.tolist()
        assert set(status) == {0, tcd.TC_ERR_DEVICE_TIMEOUT} and status[0] != 0
        rows = torch.tensor([c == 0 for c in status], device="cuda").repeat_interleave(n)
        assert not bool(((out != good).flatten(1).any(1) & rows).any())
    w.cache.attend_wait_test(False)
    assert torch.equal(w.attend(q)[0], good) and not w.status.any()
