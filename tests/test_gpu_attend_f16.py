"""Attention in f16 where one slot outweighs each of very many others, which
together still count (GPU): f16's few exponents must not lose them."""
import numpy as np
import pytest

from cache_common import compare
from gpu_common import torch_mod

pytestmark = pytest.mark.gpu


def run(tcd, n, below, d, first, page=128):
    """One token over n cached slots and itself.  One slot's score stands `below` over the others', which are equal
    but for a ripple; its value is zero, so that the output is what the others hold.  Returns output, log-sum-exp
    and what they are in 64 bits, with the sum of magnitudes over all slots."""
    torch = torch_mod()
    rng = np.random.default_rng(n)
    total = n + 1
    pages = -(-total // page)
    k = np.zeros((pages * page, d), dtype=np.float16)
    v = rng.uniform(0.5, 1.5, (pages * page, d)).astype(np.float16)
    k[:total, 1] = rng.uniform(-0.25, 0.25, total)           # (the ripple)
    at = 3 if first else total - 3
    k[at] = 0
    k[at, 0] = below
    v[at] = 0
    q = np.zeros((1, 2, d), dtype=np.float16)
    q[0, :, 0] = 1.0
    q[0, 0, 1] = 1.0                                         # (head 1 sees no ripple: its weights coincide)
    pool = torch.zeros((1, pages, 2, 1, page, d), dtype=torch.float16, device="cuda")
    pool[0, :, 0, 0] = torch.from_numpy(k.reshape(pages, page, d)).cuda()
    pool[0, :, 1, 0] = torch.from_numpy(v.reshape(pages, page, d)).cuda()
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out = torch.zeros((1, 2, d), dtype=torch.float16, device="cuda")
    lse = torch.zeros((1, 2), device="cuda")
    st = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    tcd.KvCache(pool).attend(0, torch.from_numpy(q).cuda(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                             torch.tensor([n], dtype=torch.int32, device="cuda"), table, out, 1, scale=1.0, lse=lse,
                             status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    s = q[0].astype(np.float64) @ k[:total].astype(np.float64).T
    top = s.max(axis=1, keepdims=True)
    p = np.exp(s - top)
    want = (p @ v[:total].astype(np.float64)) / p.sum(axis=1, keepdims=True)
    return (out.double().cpu().numpy()[0], lse.double().cpu().numpy()[0], want, (top[:, 0] + np.log(p.sum(axis=1))),
            np.abs(v[:total].astype(np.float64)).sum(axis=0))


@pytest.mark.parametrize("n,below,d,first", [(131072, 17.4, 64, True), (131072, 17.4, 128, False),
                                             (131072, 16.2, 128, True), (500000, 18.0, 64, False),
                                             (500000, 18.0, 128, True), (80000, 20.5, 64, True)])
def test_many_small_weights_beside_a_large_one(tcd, n, below, d, first):
    """A score here has at most two products and is below 32: with the scaling by log2(e) and the reference's
    subtraction it is off by at most 4 roundings of 64 in 32 bits.  A weight then has twice that as its relative
    error, 2^-16 for the exponential and the sums (one is added up from at most 152 parts of 30 steps, each addition
    off by 2^-24 of it: 182 of them), and half a unit (2^-11) from its rounding to f16; below 2^-21 of the largest it
    is a multiple of 2^-31 of it (a factor of 2^7 is carried), off by at most 2^-32 of the largest weight whatever
    its own size.  The sum that divides is at least the largest weight.  The output is rounded once, its own step
    below 2^-14 being 2^-24."""
    got, lse, want, want_lse, vsum = run(tcd, n, below, d, first)
    u = 2.0 ** -11
    score = 4 * 64 * 2.0 ** -24 + 2.0 ** -16
    err = (2 * score + u) * want + 2.0 ** -32 * vsum
    compare("out", got, want, err + u * (want + err) + 2.0 ** -25)
    compare("lse", lse, want_lse, 4 * 64 * 2.0 ** -24 + 2.0 ** -16 + 4 * 2.0 ** -24 * np.abs(want_lse))
    # (the tail is worth looking at: well above a unit of the output's type)
    assert want.min() > 2.0 ** -14
