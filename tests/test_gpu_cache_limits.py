"""The largest batch that the paged cache's calls declare (GPU)."""
import pytest

from gpu_common import torch_mod

pytestmark = pytest.mark.gpu


def test_the_largest_batch_appends_attends_and_compacts(tcd):
    """65,536 sequences of two drafted tokens, a page each; the second one is accepted at both ends and in between."""
    torch = torch_mod()
    b = tcd.KV_MAX_BATCH
    pool = torch.zeros((1, b, 2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")      # 256 MB
    cache = tcd.KvCache(pool)
    table = torch.arange(b, dtype=torch.int32, device="cuda")[:, None].contiguous()
    ctx = torch.zeros(b, dtype=torch.int32, device="cuda")
    cu = 2 * torch.arange(b + 1, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((2 * b, 3 * 64), generator=g, device="cuda").bfloat16()
    q = torch.zeros((2 * b, 1, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    cache.append(0, qkv, cu, ctx, table, q)
    cache.attend(0, q, cu, ctx, table, out, 2)
    # (the first of two tokens sees itself alone)
    assert torch.equal(out[0::2, 0], qkv[0::2, 128:])
    path = torch.ones((b, 1), dtype=torch.int32, device="cuda")
    n = torch.zeros(b, dtype=torch.int32, device="cuda")
    some = [0, 1, 40000, b - 2, b - 1]
    n[some] = 1
    lens = torch.full_like(n, 9)
    before = pool.clone()
    cache.compact(table, ctx, path, n, lens)
    cache.raise_on_error()
    assert torch.equal(lens, n)
    before[0, some, :, :, 0] = before[0, some, :, :, 1]
    assert torch.equal(pool, before)


def test_one_more_is_refused(tcd):
    torch = torch_mod()
    b = tcd.KV_MAX_BATCH + 1
    pool = torch.zeros((1, 2, 2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    cache = tcd.KvCache(pool)

    def ints(*shape):
        return torch.zeros(shape, dtype=torch.int32, device="cuda")

    rows = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: cache.append(0, rows.repeat(1, 3), ints(b + 1), ints(b), ints(b, 1), rows),
                 lambda: cache.attend(0, rows, ints(b + 1), ints(b), ints(b, 1), rows.clone(), 1),
                 lambda: cache.compact(ints(b, 1), ints(b), ints(b, 1), ints(b), ints(b)),
                 lambda: cache.copy_pages(ints(b), ints(b))):
        with pytest.raises(tcd.TcError) as e:
            call()
        assert e.value.name == "TC_ERR_CAPACITY"


def test_a_copy_for_every_sequence_of_the_largest_batch(tcd):
    torch = torch_mod()
    b = tcd.KV_MAX_BATCH
    g = torch.Generator(device="cuda").manual_seed(2)
    raw = torch.randint(-32768, 32768, (1, 2 * b, 2, 1, 16, 64), generator=g, device="cuda", dtype=torch.int16)
    pool = raw.clone().view(torch.bfloat16)                                            # 512 MB
    order = torch.randperm(2 * b, generator=g, device="cuda").to(torch.int32)
    src, dst = order[:b].contiguous(), order[b:].contiguous()
    cache = tcd.KvCache(pool)
    cache.copy_pages(src, dst)
    cache.raise_on_error()
    raw[:, dst.long()] = raw[:, src.long()]
    assert torch.equal(pool.view(torch.int16), raw)
