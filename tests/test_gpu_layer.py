"""A layer's step over forked sequences with the operators one after another, as a
decoder runs them (queries, keys and values; append; attention that reads the
prompt once; back onto the residual; the gated feed-forward block), against the same
step in 64 bits from each operator's own inputs, and captured into a graph."""
import numpy as np
import pytest

from cache_common import attend_bound, attend_exact, compare
from gpu_common import torch_mod
from linear_common import act_exact

pytestmark = pytest.mark.gpu

HIDDEN, WIDE, HQ, HKV, D, PAGE, PROMPT = 256, 680, 8, 2, 64, 16, 75


class Step:
    def __init__(self, tcd, dt, batch):
        torch = torch_mod()
        self.tcd, self.batch = tcd, batch
        t = {"bf16": torch.bfloat16, "f16": torch.float16}[dt]
        self.dt, self.type = dt, t
        g = torch.Generator(device="cuda").manual_seed(3)

        def normal(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * scale).to(t)

        self.normal = normal
        wide = (HQ + 2 * HKV) * D
        self.weights = {"qkv": normal(wide, HIDDEN, scale=HIDDEN ** -0.5), "bias": normal(wide, scale=0.3),
                        "out": normal(HIDDEN, HQ * D, scale=(HQ * D) ** -0.5),
                        "gate": normal(WIDE, HIDDEN, scale=HIDDEN ** -0.5), "up": normal(WIDE, HIDDEN, scale=HIDDEN ** -0.5),
                        "down": normal(HIDDEN, WIDE, scale=WIDE ** -0.5)}
        w = self.weights
        self.qkv = tcd.Linear(w["qkv"], bias=w["bias"])
        self.out = tcd.Linear(w["out"])
        self.up = tcd.Linear(w["up"], gate=w["gate"], act=tcd.ACT_SILU)
        self.down = tcd.Linear(w["down"])
        # the prompt's pages are shared, the last, partly filled one is each sequence's own
        self.pages = tcd.PagePool(8 + 2 * batch, PAGE)
        seqs = [self.pages.open()]
        self.pages.reserve(seqs[0], 0, PROMPT)
        self.cache = tcd.KvCache(normal(1, 8 + 2 * batch, 2, HKV, PAGE, D))
        seqs += [self.pages.fork(seqs[0], PROMPT) for _ in range(batch - 1)]
        ints = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
        copies = [c for s in seqs for c in self.pages.reserve(s, PROMPT, PROMPT + 1)]
        if copies:
            self.cache.copy_pages(ints([a for a, _ in copies]), ints([b for _, b in copies]))
        self.table_host = np.stack([self.pages.row(s, 24) for s in seqs])
        self.table, self.ctx = ints(self.table_host), ints([PROMPT] * batch)
        self.cu, self.groups = ints(range(batch + 1)), (ints([0, batch]), ints([PROMPT]))
        angle = torch.arange(PROMPT + 1, device="cuda")[:, None] * 1e4 ** (-torch.arange(0, D, 2, device="cuda") / D)
        self.rope = torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()
        empty = lambda n: torch.empty((batch, n), dtype=t, device="cuda")  # noqa: E731
        self.x, self.start = empty(HIDDEN), normal(batch, HIDDEN)
        self.b = {"qkv": empty(wide), "q": empty(HQ * D), "o": empty(HQ * D), "mid": empty(HIDDEN), "up": empty(WIDE)}

    def run(self):
        b = self.b
        self.x.copy_(self.start)
        self.qkv.apply(self.x, b["qkv"])
        self.cache.append(0, b["qkv"], self.cu, self.ctx, self.table, b["q"], rope=self.rope)
        self.cache.attend_shared(0, b["q"], self.cu, self.ctx, self.table, b["o"], 1, *self.groups)
        self.out.apply(b["o"], self.x, residual=self.x)
        b["mid"].copy_(self.x)
        self.up.apply(self.x, b["up"])
        self.down.apply(b["up"], self.x, residual=self.x)

    def raise_on_error(self):
        self.cache.raise_on_error()
        for x in (self.qkv, self.out, self.up, self.down):
            x.raise_on_error()


def off(got, want, mag, k, u):
    """Half a step of the type, and k products and sums in 32 bits of magnitude `mag`."""
    err = (k + 40) * 2.0 ** -23 * mag
    compare("product", got, want, err + u * (np.abs(want) + err) + 2.0 ** -25)


@pytest.mark.parametrize("batch", [3, 90])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_step(tcd, dt, batch):
    torch_mod()
    s = Step(tcd, dt, batch)
    s.run()
    s.raise_on_error()
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dt]
    w = {k: f(v) for k, v in s.weights.items()}
    b, start, x = {k: f(v) for k, v in s.b.items()}, f(s.start), f(s.x)
    off(b["qkv"], start @ w["qkv"].T + w["bias"], np.abs(start) @ np.abs(w["qkv"]).T + np.abs(w["bias"]), HIDDEN, u)
    pool, scale = f(s.cache.pool[0]), D ** -0.5
    for i in range(batch):
        n = PROMPT + 1
        kv = np.stack([pool[s.table_host[i, j // PAGE], :, :, j % PAGE] for j in range(n)], 2)   # [2, kv_heads, n, d]
        q = b["q"][i].reshape(1, HQ, D)
        want, mag, _, big = attend_exact(q, kv, np.ones((1, n), bool), scale, HQ // HKV)
        vsum = np.abs(kv[1]).sum(1).repeat(HQ // HKV, axis=0)[None]
        compare("attention", b["o"][i].reshape(1, HQ, D), want, attend_bound(dt, want, mag, big, vsum, D))
    off(b["mid"], b["o"] @ w["out"].T + start, np.abs(b["o"]) @ np.abs(w["out"]).T + np.abs(start), HQ * D, u)
    z, g = b["mid"] @ w["up"].T, b["mid"] @ w["gate"].T
    m = np.abs(b["mid"])
    a = act_exact(g, "silu")
    off(b["up"], a * z, (np.abs(a) * (m @ np.abs(w["up"]).T) + 1.13 * (m @ np.abs(w["gate"]).T) * np.abs(z)) +
        (6 + 1.2 * np.abs(g)) * np.abs(a * z) / HIDDEN, HIDDEN, u)
    off(x, b["up"] @ w["down"].T + b["mid"], np.abs(b["up"]) @ np.abs(w["down"]).T + np.abs(b["mid"]), WIDE, u)


def test_step_in_a_graph_beside_plain_calls(tcd):
    """Captured once and replayed on one stream, while steps of another batch run on a second."""
    torch = torch_mod()
    a, b = Step(tcd, "bf16", 90), Step(tcd, "f16", 5)
    a.run()
    b.run()
    torch.cuda.synchronize()
    want_a, want_b = a.x.clone(), b.x.clone()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        a.run()
    a.x.zero_()
    b.x.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s):
            g.replay()
        with torch.cuda.stream(t):
            b.run()
    torch.cuda.synchronize()
    a.raise_on_error()
    b.raise_on_error()
    assert torch.equal(a.x, want_a) and torch.equal(b.x, want_b)


def test_calls_on_a_stream_that_is_not_the_current_one(tcd):
    """The objects take the stream of the call; buffers that they own belong to it."""
    torch = torch_mod()
    s = Step(tcd, "bf16", 90)
    s.run()
    torch.cuda.synchronize()
    want = s.b["o"].clone(), s.x.clone()
    other = torch.cuda.Stream()
    out, y = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    torch.cuda.synchronize()
    s.cache.attend_shared(0, s.b["q"], s.cu, s.ctx, s.table, out, 1, *s.groups, stream=other)
    s.out.apply(out, y, residual=s.start, stream=other)
    torch.cuda.synchronize()
    s.raise_on_error()
    assert torch.equal(out, want[0]) and torch.equal(y, s.b["mid"])
