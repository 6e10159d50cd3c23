"""The order of a projection's sums follows from its sizes: where the output and the
residual lie, and how far their rows are apart, changes no bit of the results."""
import pytest

from gpu_common import torch_mod
from linear_common import ACTS, Layer

pytestmark = pytest.mark.gpu

SIZES = [(n, k, out) for n in (1, 17, 130, 200, 240, 256, 300, 400, 520, 700) for k, out in
         ((512, 1024), (1024, 512), (2048, 640), (4096, 1024), (1000, 2732), (304, 500))]


def place(like, gap, offset):
    """Rows `gap` elements wider, the first one `offset` elements from an aligned address."""
    torch = torch_mod()
    n, m = like.shape
    line = torch.full((offset + n * (m + gap) + 8,), 55.0, dtype=like.dtype, device="cuda")
    return line[offset:offset + n * (m + gap)].view(n, m + gap)[:, :m]


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_alignment_changes_no_bit(tcd, size, gate):
    torch = torch_mod()
    i = SIZES.index(size)
    w = Layer(tcd, *size, ["bf16", "f16"][i % 2], ACTS[i % 5], bias=True, gate=gate, residual=True, seed=i)
    want = w.run().clone()
    for gap, offset in ((0, 1), (3, 0), (0, 4), (4, 2), (1, 3)):
        for out, residual in ((place(want, gap, offset), w.r), (place(want, 0, 0), place(w.r, gap, offset)),
                              (place(want, gap, offset), place(w.r, 1, offset))):
            if residual is not w.r:
                residual.copy_(w.r)
            w.linear.apply(w.x, out, residual=residual)
            assert not int((out != want).sum()), (gap, offset)
    w.linear.raise_on_error()
