"""The cache object's own status and workspace buffers on several streams (GPU)."""
import pytest

torch = pytest.importorskip("torch")

from cache_common import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tcd():
    from trie_constrained_decoding_gb300 import binding
    return binding


def test_errors_on_a_side_stream_are_waited_for(tcd):
    """raise_on_error sees a code that a busy side stream has yet to write; each
    stream has buffers of its own."""
    w = Batch(tcd, [3, 2], [70, 10], "bf16", 2, 64, 16, seed=3)
    w.fill()
    q, _ = w.normal(w.n, 4, 64)
    out = torch.empty_like(q)
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 3)
    w.cache.raise_on_error()
    bad = w.ctx.clone()
    bad[1] = -1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    w.cache.attend(0, q, w.cu, bad, w.table, out, 3, stream=side)
    with pytest.raises(tcd.TcError) as e:
        w.cache.raise_on_error()
    assert e.value.code == tcd.TC_ERR_BOUNDS
    w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 3)
    w.cache.raise_on_error()


def test_outgrown_buffers_stay(tcd):
    """A graph that was captured with the object's status buffer still writes to
    memory that is its own when the buffer has grown since."""
    w = Batch(tcd, [1], [20], "bf16", 1, 64, 16, seed=5)
    w.fill()
    q, _ = w.normal(w.n, 2, 64)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 1)
    want = out.clone()
    n = 200
    with torch.cuda.stream(side):
        many = torch.full((n,), -1, dtype=torch.int32, device="cuda")  # (refused, nothing is copied)
        w.cache.copy_pages(many, many)
        filler = torch.full((1024,), 7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert bool((filler == 7).all())
