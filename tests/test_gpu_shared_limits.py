"""Attention behind shared prefixes with the declared batch of 65,536 sequences, in one
group, in as many groups as can share and in groups of one."""
import numpy as np
import pytest

from cache_common import attend_bound, attend_exact, compare
from gpu_common import torch_mod

pytestmark = pytest.mark.gpu

BATCH, PAGE, D = 65536, 16, 64


@pytest.mark.parametrize("alike", [65536, 2, 1])
@pytest.mark.parametrize("long", [False, True])
def test_most_sequences(tcd, alike, long):
    """alike: sequences of a group, which have their first page in common.  long: more rows than a short rest may have."""
    torch = torch_mod()
    heads, tokens = (65, 1) if long else (2, 1)
    g = torch.Generator(device="cuda").manual_seed(alike)
    ctx, pages = 18, 2 * BATCH
    pool = torch.randn((1, pages, 2, 1, PAGE, D), generator=g, device="cuda").bfloat16()
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = order.view(BATCH, 2).clone()
    first = torch.arange(BATCH, device="cuda") // alike * alike
    table[:, 0] = table[first, 0]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = torch.arange(BATCH + 1, device="cuda", dtype=torch.int32) * tokens
    cu_seqs = torch.arange(BATCH // alike + 1, device="cuda", dtype=torch.int32) * alike
    lens = torch.full((BATCH // alike,), PAGE + 2, dtype=torch.int32, device="cuda")
    ctx_lens = torch.full((BATCH,), ctx, dtype=torch.int32, device="cuda")
    q = torch.randn((BATCH * tokens, heads, D), generator=g, device="cuda").bfloat16()
    out, plain = torch.full_like(q, 55.0), torch.full_like(q, 55.0)
    cache = tcd.KvCache(pool)
    status = ints([7] * BATCH)
    cache.attend_shared(0, q, cu, ctx_lens, table, out, tokens, cu_seqs, lens, status=status)
    assert not bool(status.any())
    cache.attend(0, q, cu, ctx_lens, table, plain, tokens, status=status)
    assert not bool(status.any())
    most = pool[0, :, 1].float().abs().max().item()
    assert float((out.float() - plain.float()).abs().max()) <= 4 * 2.0 ** -8 * most
    for b in [0, 1, 2, 3, 511, 512, 4097, 32767, 32768, 65534, 65535]:
        kv = pool[0, table[b].long()].double().cpu().numpy().transpose(1, 2, 0, 3, 4).reshape(2, 1, 2 * PAGE, D)
        kv = kv[:, :, :ctx + tokens]
        q64 = q[b * tokens:(b + 1) * tokens].double().cpu().numpy()
        seen = np.arange(ctx + tokens)[None] <= ctx + np.arange(tokens)[:, None]
        want, mag, _, big = attend_exact(q64, kv, seen, D ** -0.5, heads)
        vsum = np.einsum("tn,hnd->thd", seen.astype(np.float64), np.abs(kv[1])).repeat(heads, axis=1)
        compare(f"sequence {b}", out[b * tokens:(b + 1) * tokens].double().cpu().numpy(), want,
                attend_bound("bf16", want, mag, big, vsum, D))
