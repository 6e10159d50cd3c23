"""Errors of calls without `status` (GPU): none is lost behind a later call that
succeeds, and each is raised once."""
import pytest

from cache_common import Batch
from gpu_common import torch_mod

pytestmark = pytest.mark.gpu


def setup(tcd, layers=2):
    torch = torch_mod()
    w = Batch(tcd, [3, 2, 4], [10, 40, 0], "bf16", 2, 64, 16, layers=layers, seed=41)
    for layer in range(layers):
        w.fill(layer)
    qkv, _ = w.normal(w.n, 8 * 64)
    q = torch.zeros((w.n, 4, 64), dtype=torch.bfloat16, device="cuda")
    return w, qkv, q, torch.zeros_like(q), torch.ones((60, 32, 2), device="cuda")


def raised(tcd, w):
    with pytest.raises(tcd.TcError) as e:
        w.cache.raise_on_error()
    w.cache.raise_on_error()       # (once)
    return e.value.name, str(e.value)


def test_an_append_that_wrote_nothing_is_reported_after_a_good_attend(tcd):
    """A position outside the angle table in the first of two layers."""
    torch = torch_mod()
    w, qkv, q, out, rope = setup(tcd)
    pos = torch.arange(w.n, dtype=torch.int32, device="cuda")
    wrong = pos.clone()
    wrong[4] = 60                                                   # a token of sequence 1
    for layer, p in enumerate((wrong, pos)):
        w.cache.append(layer, qkv, w.cu, w.ctx, w.table, q, rope=rope, positions=p)
        w.cache.attend(layer, q, w.cu, w.ctx, w.table, out, 4)
    name, text = raised(tcd, w)
    assert name == "TC_ERR_BOUNDS" and "sequence 1" in text


def test_the_first_error_of_a_sequence_stays(tcd):
    w, qkv, q, out, rope = setup(tcd)
    ctx = w.ctx.clone()
    ctx[0] = -1
    w.cache.attend(0, q, w.cu, ctx, w.table, out, 4)
    w.cache.attend_wait_test(True, 2000)
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 4)
    w.cache.attend_wait_test(False, 0)
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 4)
    assert raised(tcd, w)[0] == "TC_ERR_BOUNDS"
    w.cache.attend_wait_test(True, 2000)
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 4)
    w.cache.attend_wait_test(False, 0)
    w.cache.attend(0, q, w.cu, ctx, w.table, out, 4)
    assert raised(tcd, w)[0] == "TC_ERR_DEVICE_TIMEOUT"


def test_copies_and_compaction_are_reported(tcd):
    torch = torch_mod()
    w, qkv, q, out, rope = setup(tcd)

    def ints(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    w.cache.copy_pages(ints(*[-1] * 70, 0), ints(*range(71)))      # (more pairs than sequences)
    w.cache.copy_pages(ints(0), ints(1))
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 4)
    name, text = raised(tcd, w)
    assert name == "TC_ERR_BOUNDS" and "page copy 0" in text
    lens = torch.zeros_like(w.ctx)
    w.cache.compact(w.table, w.ctx, ints(0, 1, 1, 0, 0, 1).view(3, 2), ints(2, 2, 2), lens)
    w.cache.compact(w.table, w.ctx, ints(0, 1, 0, 1, 0, 1).view(3, 2), ints(2, 2, 2), lens)
    name, text = raised(tcd, w)
    assert name == "TC_ERR_BOUNDS" and "sequence 1" in text


def test_a_replay_does_not_clear_the_error_of_the_one_before(tcd):
    torch = torch_mod()
    w, qkv, q, out, rope = setup(tcd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        w.cache.append(0, qkv, w.cu, w.ctx, w.table, q, rope=rope)
        w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 4)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        w.cache.append(0, qkv, w.cu, w.ctx, w.table, q, rope=rope)
        w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 4)
    good = w.ctx.clone()
    g.replay()
    w.cache.raise_on_error()
    w.ctx[2] = 57                                                  # (past the angle table: 60 positions)
    g.replay()
    w.ctx.copy_(good)
    g.replay()
    g.replay()
    name, text = raised(tcd, w)
    assert name == "TC_ERR_BOUNDS" and "sequence 2" in text


def test_a_given_status_is_written_whole(tcd):
    torch = torch_mod()
    w, qkv, q, out, rope = setup(tcd)
    ctx = w.ctx.clone()
    ctx[1] = -5
    st = torch.full((3,), 99, dtype=torch.int32, device="cuda")
    w.cache.attend(0, q, w.cu, ctx, w.table, out, 4, status=st)
    assert st.tolist() == [0, tcd.TC_ERR_BOUNDS, 0]
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 4, status=st)
    assert st.tolist() == [0, 0, 0]
    w.cache.raise_on_error()
