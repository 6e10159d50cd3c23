"""Waits that are much too short for the work: a call says that it gave up or is
right, and what it had begun does not reach into later calls."""
import numpy as np
import pytest

from cache_common import Batch
from gpu_common import torch_mod
from linear_common import Layer
from test_gpu_attend_shared import Groups

pytestmark = pytest.mark.gpu

POLLS = [1, 2, 3, 5, 8, 20, 60, 200]


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("size", [(1, 2048, 512), (64, 3000, 600), (300, 1000, 520), (1500, 2000, 1030)], ids=str)
def test_projections(tcd, size, gate):
    torch = torch_mod()
    w = Layer(tcd, *size, gate=gate, bias=True, residual=True, seed=4)
    good = w.run().clone()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for polls in POLLS:
        for _ in range(3):
            word.zero_()
            w.y.fill_(w.MARK)
            w.linear.wait_test(False, polls)
            w.linear.apply(w.x, w.y, residual=w.r, status=word)
            if word.item() == 0:
                assert torch.equal(w.y, good)
            else:
                assert word.item() == tcd.TC_ERR_DEVICE_TIMEOUT
            w.linear.wait_test(False, 0)
            assert torch.equal(w.run(), good)


@pytest.mark.parametrize("d", [64, 128])
def test_attention(tcd, d):
    torch = torch_mod()
    w = Batch(tcd, [1, 300, 7, 1], [500, 0, 2000, 40], "bf16", 2, d, 32, seed=2)
    w.fill()
    q, _ = w.normal(w.n, 8, d)
    out, good = torch.empty_like(q), torch.empty_like(q)
    w.cache.attend(0, q, w.cu, w.ctx, w.table, good, 300, status=w.status)
    for polls in POLLS:
        for _ in range(3):
            w.cache.attend_wait_test(False, polls)
            out.fill_(55)
            w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 300, status=w.status)
            status = w.status.tolist()
            assert status in ([0] * 4, [tcd.TC_ERR_DEVICE_TIMEOUT] * 4)
            assert any(status) or torch.equal(out, good)
            w.cache.attend_wait_test(False)
            w.cache.attend(0, q, w.cu, w.ctx, w.table, out, 300, status=w.status)
            assert not w.status.any() and torch.equal(out, good)


# heads of a group, head_dim, tokens of a sequence
RESTS = [(16, 128, 4), (32, 128, 2), (16, 64, 4), (4, 64, 13), (1, 128, 64), (64, 64, 1)]


@pytest.mark.parametrize("only_rests", [True, False])
@pytest.mark.parametrize("case", range(len(RESTS)))
def test_shared_prefixes(tcd, case, only_rests):
    """Items of up to 64 rows, half of them with rows in two warps' hands; sequences with nothing wrong have the same
    bits as always."""
    torch = torch_mod()
    group, d, n = RESTS[case]
    rng = np.random.default_rng(case)
    tokens = [int(x) for x in rng.choice([n, max(1, n // 2)], 200)]
    w = Groups(tcd, tokens, [int(x) for x in 48 + rng.integers(0, 300, 200)], [(0, 90, 48), (90, 200, 32)], "bf16", 4, d, 16,
               7, heads=group)
    w.fill()
    q, _ = w.normal(w.n, 4 * group, d)
    good = w.attend(q)[0].clone()
    assert not w.status.any()
    need = w.cache.shared_workspace_bytes(w.n, 4 * group)
    ws = torch.empty((need + 3) // 4, dtype=torch.int32, device="cuda")
    counts = torch.tensor(tokens, device="cuda")
    seen = set()
    for polls in POLLS:
        for _ in range(6):
            w.cache.attend_wait_test(2 if only_rests else 0, polls)
            ws.view(torch.float32).fill_(1.0)       # (as another call has left it: every row's own part is there)
            ws[-(w.n * 4 * group + 64):] = 1
            out, _ = w.attend(q, workspace=ws)
            status = w.status.tolist()
            seen |= set(status)
            right = torch.tensor([c == 0 for c in status], device="cuda").repeat_interleave(counts)
            wrong = (out != good).flatten(1).any(1) & right
            assert not bool(wrong.any()), (polls, int(wrong.sum()))
            w.cache.attend_wait_test(False)
            assert torch.equal(w.attend(q, workspace=ws)[0], good) and not w.status.any()
    assert seen <= {0, tcd.TC_ERR_DEVICE_TIMEOUT}
