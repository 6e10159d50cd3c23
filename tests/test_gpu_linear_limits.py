"""Projections of the largest sizes that a call takes, in one direction each."""
import pytest

from gpu_common import torch_mod

pytestmark = pytest.mark.gpu

SIZES = [(1 << 24, 8, 8), ((1 << 24) - 3, 5, 3), (1, 1 << 20, 8), (3, (1 << 20) - 7, 5), (300, 1 << 20, 16),
         (5, 8, 1 << 20), (200, 16, (1 << 20) - 1), (1500, 24, 1 << 20)]


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_largest(tcd, size, gate):
    """Small whole numbers: every sum is exact in 32 bits in any order, and so is what it is rounded to."""
    torch = torch_mod()
    n, k, out = size
    g = torch.Generator(device="cuda").manual_seed(n + out)

    def rows(m, cols, most):
        wide = -(-cols // 8) * 8
        v = torch.randint(-most, most + 1, (m, wide), generator=g, device="cuda", dtype=torch.int8).bfloat16()
        return v[:, :cols]

    most = 1 if k > 1000 else 2
    x, w, v = rows(n, k, most), rows(out, k, most), rows(out, k, most) if gate else None
    if k > 1000:                       # (so that sums stay below 2^24, and with a gate products)
        x[:, 3000:] = 0
    residual = rows(n, out, 3)
    y = torch.full((n, out), 55.0, dtype=x.dtype, device="cuda")
    linear = tcd.Linear(w, gate=v, act=tcd.ACT_RELU)
    linear.apply(x, y, residual=residual)
    linear.raise_on_error()
    used = min(k, 3000)
    w32, v32 = w[:, :used].float(), None if v is None else v[:, :used].float()
    step = max(1, (1 << 28) // out)
    for i in range(0, n, step):
        part = x[i:i + step, :used].float()
        z = part @ w32.T               # (exact as well, in this type)
        if gate:
            z = (part @ v32.T).clamp(min=0) * z
        else:
            z = z.clamp(min=0)
        want = (z + residual[i:i + step].to(z.dtype)).to(y.dtype)
        assert torch.equal(y[i:i + step], want), i
