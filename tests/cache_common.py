"""Shared by the GPU tests of the paged cache: ragged batches with scattered
pages, and the operators' definitions in 64 bits (numpy, on the host)."""
from __future__ import annotations

import numpy as np

from gpu_common import torch_mod

# Half the distance of neighbouring numbers, relative: 8 and 11 significant bits.
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def dtype(name):
    torch = torch_mod()
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


class Batch:
    """Sequences of `tokens[b]` new tokens behind `ctx[b]` cached ones, their pages scattered over the pool.

    Every page that no sequence holds, and every slot past a sequence's last one, holds NaN."""

    def __init__(self, tcd, tokens, ctx, dt="bf16", kv_heads=2, head_dim=128, page=16, layers=1, seed=0, spare=3,
                 extra_width=2):
        torch = torch_mod()
        self.rng = np.random.default_rng(seed)
        self.tokens, self.ctx_list, self.dt, self.page = list(tokens), list(ctx), dt, page
        self.kv_heads, self.head_dim, self.layers = kv_heads, head_dim, layers
        need = [-(-(t + c) // page) for t, c in zip(tokens, ctx)]
        self.pages = sum(need) + spare
        order = self.rng.permutation(self.pages)
        width = max(max(need), 1) + extra_width
        self.table_host = np.full((len(tokens), width), -7, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table_host[b, :n] = order[at:at + n]
            at += n
        self.n = sum(self.tokens)
        self.cu_host = np.concatenate(([0], np.cumsum(self.tokens))).astype(np.int32)
        self.pool = torch.full((layers, self.pages, 2, kv_heads, page, head_dim), float("nan"), dtype=dtype(dt),
                               device="cuda")
        self.cu = torch.from_numpy(self.cu_host).cuda()
        self.ctx = torch.tensor(self.ctx_list, dtype=torch.int32, device="cuda")
        self.table = torch.from_numpy(self.table_host).cuda()
        self.status = torch.full((len(tokens),), 77, dtype=torch.int32, device="cuda")
        self.cache = tcd.KvCache(self.pool)

    def normal(self, *shape):
        """Normal values on the device, and what they are in 64 bits."""
        torch = torch_mod()
        t = torch.from_numpy(self.rng.standard_normal(shape, dtype=np.float32)).to(dtype(self.dt)).cuda()
        return t, t.double().cpu().numpy()

    def slots(self, b, lo, hi):
        """(page, offset) of slots [lo, hi) of sequence b."""
        s = np.arange(lo, hi)
        return self.table_host[b, s // self.page], s % self.page

    def fill(self, layer=0, scale=1.0):
        """Keys and values for every slot of every sequence; returns them in 64 bits per sequence [2, kv_heads, n, d]."""
        torch = torch_mod()
        got = []
        for b, (t, c) in enumerate(zip(self.tokens, self.ctx_list)):
            dev, host = self.normal(2, self.kv_heads, t + c, self.head_dim)
            if scale != 1.0:
                dev = (dev.float() * scale).to(dev.dtype)
                host = dev.double().cpu().numpy()
            pages, offs = self.slots(b, 0, t + c)
            if t + c:
                self.pool[layer, torch.from_numpy(pages).long().cuda(), :, :, torch.from_numpy(offs).cuda()] = \
                    dev.permute(2, 0, 1, 3)
            got.append(host)
        return got

    def seen(self, masks=None):
        """Per sequence, [tokens, slots]: what each token sees (causal, or the tree's bits as Python ints)."""
        out = []
        for b, (t, c) in enumerate(zip(self.tokens, self.ctx_list)):
            m = np.zeros((t, t + c), dtype=bool)
            m[:, :c] = True
            for i in range(t):
                for j in range(t):
                    m[i, c + j] = (j <= i) if masks is None else bool(masks[self.cu_host[b] + i] >> j & 1)
            out.append(m)
        return out


def attend_exact(q, kv, seen, scale, group):
    """Output, sum_j p_j |v_j|, log-sum-exp and largest score sums of one sequence, in 64 bits.

    q [t, heads, d], kv [2, kv_heads, n, d], seen [t, n]."""
    t, heads, d = q.shape
    out, mag, lse = np.zeros((t, heads, d)), np.zeros((t, heads, d)), np.full((t, heads), -np.inf)
    big = np.zeros((t, heads))
    for h in range(heads):
        k, v = kv[0, h // group], kv[1, h // group]
        for i in range(t):
            use = seen[i]
            if not use.any():
                continue
            s = k[use] @ q[i, h] * scale
            big[i, h] = (np.abs(k[use]) @ np.abs(q[i, h])).max() * abs(scale)
            top = s.max()
            p = np.exp(s - top)
            lse[i, h] = top + np.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ v[use]
            mag[i, h] = p @ np.abs(v[use])
    return out, mag, lse, big


def attend_bound(dt, out, mag, big, vsum, d):
    """Largest error of an element.

    A score is a sum of d exact products in 32 bits: it is off by at most
    d 2^-24 times the sum of their magnitudes, and the scaling and the
    subtraction of the maximum add as much as 4 more roundings of it.  A weight
    (and the sum that divides it) then has a relative error of twice that, plus
    2^-21 for the exponential and the running sums, plus the rounding of the
    weight to the cache's type.  f16 has no weights below 2^-24: an absolute
    error of 2^-25 for each slot (`vsum`: sum of |v| over the slots seen).  The
    output is rounded once."""
    u = UNIT[dt]
    score = 2 * (d + 4) * 2.0 ** -24 * big[..., None] + 2.0 ** -21
    tiny = 2.0 ** -25 * vsum if dt == "f16" else 0.0
    err = (2 * score + u) * mag + tiny
    return err + u * (np.abs(out) + err) + 1e-30


def compare(what, got, want, bound):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0].tolist(), float(got[bad][0]), float(want[bad][0]),
                           float(np.broadcast_to(bound, want.shape)[bad][0]))


def ancestors(parents):
    words = []
    for i, p in enumerate(parents):
        words.append((words[p] if p >= 0 else 0) | 1 << i)
    return words


def random_parents(rng, n):
    return [-1 if i == 0 or rng.random() < 0.15 else int(rng.integers(max(0, i - 5), i)) for i in range(n)]


def mask_words(masks, words):
    """Python integers to int64 [n, words] on the device."""
    torch = torch_mod()
    w = np.array([[(m >> 64 * k) & (1 << 64) - 1 for k in range(words)] for m in masks], dtype=np.uint64)
    return torch.from_numpy(w.reshape(len(masks), words).view(np.int64)).cuda()
