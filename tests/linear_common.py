"""Shared by the GPU tests of the projections: the definition in 64 bits (numpy,
on the host) and how far a result may be from it."""
from __future__ import annotations

import math

import numpy as np

from cache_common import UNIT, dtype
from gpu_common import torch_mod

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act_exact(z, act):
    with np.errstate(over="ignore"):
        if act == "relu":
            return np.maximum(z, 0)
        if act == "silu":
            return z / (1 + np.exp(-z))
        if act == "gelu":
            return z / 2 * _erfc(-z / math.sqrt(2))
        if act == "gelu_tanh":
            return z / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def act_error(z, dz, act):
    """Of a value that is off by dz: dz times the largest slope (1.13), and the activation's own error in 32 bits.

    silu: an exponential (2 + 1.173 |z| units of 2^-23), a sum and a division (2 units); gelu_tanh: the same for an
    exponent of 2 u that is itself off by 4 units; gelu: erfc of an argument that is off by 2 units (the logarithm's slope
    is at most 2 |z / sqrt 2| + 2 there) with 4 units of its own, and two products."""
    a = np.abs(act_exact(z, act))
    if act in ("none", "relu"):
        return dz
    if act == "silu":
        own = 6 + 1.2 * np.abs(z)
    elif act == "gelu_tanh":
        own = 6 + 5.2 * 2 * math.sqrt(2 / math.pi) * (np.abs(z) + 0.044715 * np.abs(z) ** 3)
    else:
        own = 8 + 2 * (z * z + 2 * np.abs(z))
    # (below 2^-126 results are flushed to zero)
    return 1.13 * dz + 2.0 ** -23 * own * a + 2.0 ** -126 * (1 + np.abs(z))


class Layer:
    """Weights and inputs of one projection, as tensors and in 64 bits.  Rows of x, out and the residual are slices
    of wider ones; what lies beside them holds NaN (inputs) or a mark (out)."""

    MARK = 55.0

    def __init__(self, tcd, n, k, out, dt="bf16", act="none", bias=False, gate=False, residual=False, gap=0, seed=0,
                 whole=False):
        torch = torch_mod()
        rng = np.random.default_rng(seed)
        self.tcd, self.n, self.k, self.features, self.dt, self.act = tcd, n, k, out, dt, act
        t = dtype(dt)

        def rows(m, cols, stride, scale):
            """[m, cols] within rows of `stride` elements."""
            v = rng.integers(-3, 4, (m, cols)).astype(np.float32) if whole else \
                rng.standard_normal((m, cols), dtype=np.float32) * np.float32(scale)
            big = torch.full((m, stride), float("nan"), dtype=t, device="cuda")
            big[:, :cols] = torch.from_numpy(v).to(t).cuda()
            return big[:, :cols], big[:, :cols].double().cpu().numpy()

        wide = -(-k // 8) * 8
        self.x, self.x64 = rows(n, k, wide + 8 * gap, 1.0)
        self.w, self.w64 = rows(out, k, wide + 8 * (gap & 1), k ** -0.5)
        self.v, self.v64 = rows(out, k, wide, 1.5 * k ** -0.5) if gate else (None, None)
        self.b, self.b64 = rows(1, out, out, 0.5) if bias else (None, 0.0)
        self.c, self.c64 = rows(1, out, out, 0.5) if bias and gate else (None, 0.0)
        self.r, self.r64 = rows(n, out, out + gap, 2.0) if residual else (None, 0.0)
        self.big = torch.full((n + 2, out + gap), self.MARK, dtype=t, device="cuda")
        self.y = self.big[1:n + 1, :out]
        self.linear = tcd.Linear(self.w, bias=None if self.b is None else self.b[0], gate=self.v,
                                 gate_bias=None if self.c is None else self.c[0], act=getattr(tcd, "ACT_" + act.upper()))

    def run(self, **kw):
        torch_mod()
        self.linear.apply(self.x, self.y, residual=self.r, **kw)
        self.linear.raise_on_error()
        return self.y

    def exact(self):
        """The result, and the largest error before it is rounded.

        A sum of k exact products in 32 bits is off by at most (k + 20) 2^-23 of the sum of their magnitudes (an addition may
        truncate; 20 covers the parts that are added and the bias)."""
        per = (self.k + 20) * 2.0 ** -23
        z = self.x64 @ self.w64.T + self.b64
        dz = per * (np.abs(self.x64) @ np.abs(self.w64).T + np.abs(self.b64))
        if self.v is None:
            y, dy = act_exact(z, self.act), act_error(z, dz, self.act)
        else:
            g = self.x64 @ self.v64.T + self.c64
            dg = act_error(g, per * (np.abs(self.x64) @ np.abs(self.v64).T + np.abs(self.c64)), self.act)
            a = act_exact(g, self.act)
            y = a * z
            dy = np.abs(a) * dz + dg * (np.abs(z) + dz) + 2.0 ** -23 * np.abs(y)
        return y + self.r64, dy + 2.0 ** -23 * (np.abs(y) + np.abs(self.r64))

    def check(self):
        torch = torch_mod()
        want, err = self.exact()
        got = self.y.double().cpu().numpy()
        u = UNIT[self.dt]
        # (half a step of the type, which is constant below its smallest normal number)
        bound = err + u * (np.abs(want) + err) + (2.0 ** -25 if self.dt == "f16" else 2.0 ** -134)
        bad = ~(np.abs(got - want) <= bound)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist(), got[bad][0], want[bad][0], bound[bad][0])
        rest = self.big.clone()
        rest[1:self.n + 1, :self.features] = self.MARK
        assert bool((rest == self.MARK).all()), "written outside of out"
        assert torch.isfinite(self.y).all()
