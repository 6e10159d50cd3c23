"""Attention where a call leaves the usual path (GPU): outputs that allow only
16-byte stores, and infinities and NaN in values that the two row tiles of an item
share."""
import pytest

from cache_common import Batch, ancestors, mask_words, random_parents
from gpu_common import torch_mod

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dt", [(64, "bf16"), (64, "f16"), (128, "bf16"), (128, "f16")])
@pytest.mark.parametrize("offset,extra", [(8, 16), (0, 8), (24, 40)])
def test_outputs_aligned_to_16_bytes_only(tcd, d, dt, offset, extra):
    """The same bits as with aligned rows, in whole items, items of two row tiles and items that are cut; nothing
    between the rows is touched."""
    torch = torch_mod()
    w = Batch(tcd, [3, 150, 1, 20], [40, 700, 6000, 0], dt, 2, d, 32, seed=61)
    w.fill()
    q, _ = w.normal(w.n, 6, d)
    want = torch.zeros_like(q)
    w.cache.attend(0, q, w.cu, w.ctx, w.table, want, 150, status=w.status)
    wide = 6 * d + max(extra, offset)
    if wide % 16 == 0 and offset % 16 == 0:
        wide += 8
    buf = torch.full((w.n, wide), 55.0, dtype=q.dtype, device="cuda")
    out = buf[:, offset:offset + 6 * d]
    assert out.data_ptr() % 32 or out.stride(0) % 16
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 150, status=w.status)
    torch.cuda.synchronize()
    assert w.status.tolist() == [0] * 4
    assert torch.equal(out.reshape(w.n, 6, d), want)
    assert (buf[:, :offset] == 55).all() and (buf[:, offset + 6 * d:] == 55).all()


@pytest.mark.parametrize("d,dt", [(64, "bf16"), (64, "f16"), (128, "bf16"), (128, "f16")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("which", [0, 1])
def test_what_is_not_seen_does_not_count_in_two_row_tiles(tcd, d, dt, bad, which):
    """Drafted tokens of other branches and later tokens of a prompt, in either half of a row, one of them seen from
    the second row tile only."""
    torch = torch_mod()
    w = Batch(tcd, [150, 80], [61, 130], dt, 2, d, 16, seed=67)
    w.fill()
    q, _ = w.normal(w.n, 4, d)                       # (64 tokens a row tile)
    masks = [m for n in w.tokens for m in ancestors(random_parents(w.rng, n))]
    tree = mask_words(masks, 3)

    def run(tree=None):
        out, lse = torch.full_like(q, 55.0), torch.zeros((w.n, 4), device="cuda")
        w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 150, tree=tree, lse=lse, status=w.status)
        torch.cuda.synchronize()
        assert w.status.tolist() == [0, 0]
        return out, lse

    clean = {True: run(tree), False: run()}
    spots = ((0, 100, 2, 9), (0, 7, d - 11, d), (1, 3, 30, 35))   # sequence, token, elements
    for b, at, lo, hi in spots:
        pages, offs = w.slots(b, w.ctx_list[b] + at, w.ctx_list[b] + at + 1)
        w.pool[0, int(pages[0]), which, :, int(offs[0]), lo:hi] = bad
    for drafted in (True, False):
        out, lse = run(tree if drafted else None)
        for b in range(2):
            for i in range(w.tokens[b]):
                r = w.cu_host[b] + i
                hit = [(lo, hi) for s, at, lo, hi in spots if s == b and
                       (masks[r] >> at & 1 if drafted else at <= i)]
                old, old_lse = (x[r] for x in clean[drafted])
                if not hit:
                    assert torch.equal(out[r], old) and torch.equal(lse[r], old_lse), (drafted, b, i)
                elif which == 1:
                    touched = torch.zeros(d, dtype=torch.bool, device="cuda")
                    for lo, hi in hit:
                        touched[lo:hi] = True
                    g = out[r].float()
                    assert torch.equal(out[r][:, ~touched], old[:, ~touched]), (drafted, b, i)
                    assert torch.equal(lse[r], old_lse)
                    assert (g[:, touched].isnan() if bad != bad else g[:, touched] == bad).all(), (drafted, b, i)
                elif bad != bad:
                    assert out[r].float().isnan().all(), (drafted, b, i)
