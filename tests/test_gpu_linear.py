"""Projections against their definition in 64 bits: one token to many, odd sizes
and strides, every activation, gates, biases and residuals; sums that are exact;
infinities and NaN; the refusals."""
import numpy as np
import pytest

from gpu_common import torch_mod
from linear_common import ACTS, Layer

pytestmark = pytest.mark.gpu

SIZES = [
    # tokens, in, out, gap
    (1, 1, 1, 0), (1, 8, 4, 0), (1, 64, 128, 0), (1, 2048, 260, 0), (1, 1000, 64, 3), (2, 7, 3, 1), (3, 65, 129, 0),
    (15, 200, 127, 0), (16, 128, 128, 4), (17, 63, 65, 2), (33, 520, 300, 0), (64, 1024, 192, 16), (65, 72, 66, 0),
    (100, 333, 130, 5), (128, 256, 512, 0), (129, 320, 96, 0), (200, 4100, 70, 0), (255, 64, 257, 1),
    (256, 192, 100, 0), (257, 128, 128, 8), (300, 1000, 333, 0), (513, 96, 520, 4), (700, 640, 384, 0),
    (1030, 200, 140, 1), (140, 2048, 132, 0), (190, 700, 1030, 0), (250, 3000, 1001, 0), (300, 2500, 600, 0),
    (450, 1500, 257, 0), (600, 1300, 2050, 0), (900, 700, 4100, 0), (1300, 300, 5001, 0), (2100, 136, 9000, 0),
    (2049, 400, 1999, 0),
]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_plain_product(tcd, size, dt):
    n, k, out, gap = size
    w = Layer(tcd, n, k, out, dt, gap=gap, seed=n + k)
    w.run()
    w.check()


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_epilogue(tcd, size, gate):
    """Bias, activation, gate and residual; the activation and the type change from size to size."""
    n, k, out, gap = size
    i = SIZES.index(size)
    w = Layer(tcd, n, k, out, ["bf16", "f16"][i % 2], ACTS[i % 5], bias=True, gate=gate, residual=True, gap=gap, seed=i)
    w.run()
    w.check()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n", [3, 400])
def test_activations(tcd, act, gate, dt, n):
    """Each activation over a wide range of values: some rows are large."""
    w = Layer(tcd, n, 72, 136, dt, act, gate=gate, seed=7)
    w.x[::3] *= 9
    w.x64 = w.x.double().cpu().numpy()
    w.run()
    w.check()


EXACT = [(1, 14336, 64), (5, 4096, 130), (64, 5000, 256), (256, 1024, 128), (300, 2048, 192), (1000, 1000, 1000)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("size", EXACT, ids=str)
def test_whole_numbers_are_exact(tcd, size, gate, dt):
    """Sums of small whole numbers are exact in 32 bits in any order: the result is the rounded exact one.

    (With a gate: products below 2^24, so that they are exact as well.)"""
    torch = torch_mod()
    n, k, out = size
    if gate:
        k = min(k, 400)
    w = Layer(tcd, n, k, out, dt, "relu", bias=True, gate=gate, residual=True, seed=k, whole=True)
    y = w.run()
    want, _ = w.exact()
    assert np.abs(want).max() < 2 ** 24
    assert torch.equal(y, torch.from_numpy(want).to(y.dtype).cuda())


def test_same_bits_each_time_and_in_place(tcd):
    """Parts of a sum are added in a fixed order; the residual may be the output itself."""
    torch = torch_mod()
    for n in (1, 64, 300, 2000):
        w = Layer(tcd, n, 2048, 256, residual=True, seed=n)
        first = w.run().clone()
        for _ in range(3):
            assert torch.equal(w.run(), first)
        w.y.copy_(w.r)
        w.linear.apply(w.x, w.y, residual=w.y)
        assert torch.equal(w.y, first)


def test_infinities_and_nan_stay_in_their_rows_and_columns(tcd):
    torch = torch_mod()
    for n in (5, 300):
        w = Layer(tcd, n, 100, 140, seed=1)
        clean = w.run().clone()
        w.x[2, 50] = float("inf")
        w.w[77, 3] = float("nan")
        y = w.run()
        keep = torch.ones_like(clean, dtype=torch.bool)
        keep[2], keep[:, 77] = False, False
        assert torch.equal(y[keep], clean[keep])
        assert bool(y[:, 77].isnan().all()) and not bool(y[2].isfinite().any())


def test_no_tokens(tcd):
    torch = torch_mod()
    w = Layer(tcd, 4, 64, 32)
    w.linear.apply(w.x[:0], w.y[:0])
    torch.cuda.synchronize()
    assert bool((w.big == w.MARK).all())


@pytest.mark.parametrize("n", [1, 64, 300, 1100])
def test_wait_that_runs_out(tcd, n):
    """A load that is left out: the kernel gives up and says so, and the next call works."""
    torch = torch_mod()
    w = Layer(tcd, n, 2048, 256, seed=2)
    good = w.run().clone()
    w.linear.wait_test(True, 2000)
    w.linear.apply(w.x, w.y)
    with pytest.raises(tcd.TcError) as e:
        w.linear.raise_on_error()
    assert e.value.code == tcd.TC_ERR_DEVICE_TIMEOUT
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    w.linear.apply(w.x, w.y, status=word)
    assert word.item() == tcd.TC_ERR_DEVICE_TIMEOUT
    w.linear.wait_test(False, 0)
    assert torch.equal(w.run(), good)


def test_streams_and_graphs(tcd):
    """Two graphs of one object side by side and beside plain calls, on streams of their own."""
    torch = torch_mod()
    w = Layer(tcd, 64, 4096, 512, bias=True, seed=3)
    want = w.run().clone()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(want) for _ in range(3)]
    graphs = []
    for s, o in zip(streams[:2], outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            w.linear.apply(w.x, o)
        graphs.append(g)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        w.linear.apply(w.x, outs[2], stream=streams[2])
    torch.cuda.synchronize()
    w.linear.raise_on_error()
    for o in outs:
        assert torch.equal(o, want)


def test_refusals(tcd):
    """Arguments that a call cannot take launch nothing."""
    torch = torch_mod()
    w = Layer(tcd, 4, 64, 32)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        tcd.Linear(z(4, 8, dt=torch.float32))
    with pytest.raises(ValueError):
        tcd.Linear(z(4, 8), bias=z(5))
    with pytest.raises(ValueError):
        tcd.Linear(z(4, 8), gate=z(4, 16))
    with pytest.raises(ValueError):
        tcd.Linear(z(4, 8), gate_bias=z(4))
    with pytest.raises(ValueError):
        tcd.Linear(z(8, 4).T)
    for x, y, r in ((z(4, 63), w.y, None), (w.x, z(5, 32), None), (w.x, z(4, 31), None), (w.x, w.y, z(3, 32)),
                    (w.x, z(4, 32, dt=torch.float16), None), (w.x.cpu(), w.y, None)):
        with pytest.raises(ValueError):
            w.linear.apply(x, y, residual=r)
    odd = tcd.Linear(z(4, 9))                                # rows of 9 elements: not a multiple of 8
    for layer, x in ((odd, z(4, 9)), (w.linear, z(4, 65)[:, 1:]), (w.linear, z(4 * 64 + 8)[1:257].view(4, 64))):
        with pytest.raises(tcd.TcError) as e:
            layer.apply(x, z(4, layer.out_features))
        assert e.value.code == 1
    with pytest.raises(tcd.TcError):
        tcd.Linear(z(4, 8), act=9).apply(z(1, 8), z(1, 4))
    torch.cuda.synchronize()
    assert bool((w.big == w.MARK).all())


def test_rows_far_apart(tcd):
    """Offsets of rows beyond 2^31 elements, few tokens and many."""
    torch = torch_mod()
    for n, stride in ((100, 1 << 25), (40000, 1 << 17)):
        w = Layer(tcd, n, 64, 64, residual=True, seed=9)
        w.run()
        w.check()
        big = torch.empty((n, stride), dtype=w.y.dtype, device="cuda")
        big[:, :64] = w.r
        w.linear.apply(w.x, big[:, :64], residual=big[:, :64])
        w.linear.raise_on_error()
        assert torch.equal(big[:, :64], w.y)
        del big
        torch.cuda.empty_cache()


def test_made_and_dropped_while_a_graph_is_captured(tcd):
    """An object whose error word is new memory in the middle of a capture, and a graph that outlives its objects."""
    torch = torch_mod()
    w = Layer(tcd, 33, 256, 192, bias=True, seed=4)
    want = w.run().clone()
    s, out = torch.cuda.Stream(), torch.zeros_like(want)
    words = dict(tcd._words)
    tcd._words.clear()                                     # (the next object needs new memory)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tcd.Linear(w.w, bias=w.b[0]).apply(w.x, out)
    tcd._words.update(words)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_one_object_from_two_threads(tcd):
    import threading
    torch = torch_mod()
    layers = [Layer(tcd, n, 1024, 320, bias=True, seed=n) for n in (3, 500)]
    one = layers[0].linear
    ins = [layers[0].x, torch.randn((500, 1024), device="cuda").to(layers[0].x.dtype)]
    want = []
    for x in ins:
        y = torch.empty((x.shape[0], 320), dtype=x.dtype, device="cuda")
        one.apply(x, y)
        want.append(y)
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        y = torch.empty_like(want[i])
        s.synchronize()
        for _ in range(300):
            one.apply(ins[i], y, stream=s)
        s.synchronize()
        if not torch.equal(y, want[i]):
            bad.append(i)

    threads = [threading.Thread(target=work, args=(i % 2,)) for i in range(4)]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    one.raise_on_error()
    assert not bad
