"""tc_linear's checks of its arguments (CPU: a refused call touches no device)."""
import ctypes

import pytest

INVALID, CAPACITY, UNSUPPORTED, CUDA = 1, 10, 11, 32
AT = 1 << 20   # (an address that is never read)


CALL = ("n_tokens", "x", "x_stride", "residual", "residual_stride", "out", "out_stride", "wait_polls", "withhold")


def layer(tcd, **kw):
    v = dict(device=0, dtype=0, in_features=64, out_features=32, weight=AT, weight_stride=64, gate=None, gate_stride=0,
             bias=None, gate_bias=None, act=0)
    v.update(kw)
    return tcd._LinearWeights(*[v[n] for n, _ in tcd._LinearWeights._fields_])


def call(tcd, **kw):
    v = dict(n_tokens=4, x=AT, x_stride=64, residual=None, residual_stride=0, out=AT, out_stride=32, wait_polls=0,
             withhold=0)
    v.update(kw)
    return tcd._pack_call(*[v[n] or 0 for n in CALL])


WEIGHTS = [
    (dict(device=-1), INVALID), (dict(device=64), INVALID), (dict(in_features=0), INVALID),
    (dict(out_features=0), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(in_features=(1 << 20) + 1, weight_stride=1 << 21), CAPACITY), (dict(out_features=(1 << 20) + 1), CAPACITY),
    (dict(weight=None), INVALID), (dict(weight=AT + 8), INVALID), (dict(weight_stride=63), INVALID),
    (dict(weight_stride=56), INVALID), (dict(gate=AT + 2, gate_stride=64), INVALID), (dict(gate=AT), INVALID),
    (dict(gate=AT, gate_stride=68), INVALID), (dict(gate_bias=AT), INVALID), (dict(bias=AT + 1), INVALID),
    (dict(gate=AT, gate_stride=64, gate_bias=AT + 1), INVALID),
]
CALLS = [
    (dict(n_tokens=-1), INVALID), (dict(n_tokens=(1 << 24) + 1), CAPACITY), (dict(x=None), INVALID),
    (dict(x=AT + 2), INVALID), (dict(x_stride=60), INVALID), (dict(x_stride=56), INVALID), (dict(out=None), INVALID),
    (dict(out=AT + 1), INVALID), (dict(out_stride=31), INVALID), (dict(residual=AT, residual_stride=31), INVALID),
    (dict(residual=AT + 1, residual_stride=32), INVALID),
]


@pytest.mark.parametrize("change,code", WEIGHTS, ids=str)
def test_weights(tcd, change, code):
    assert tcd._linear(layer(tcd, **change), call(tcd), AT, None) == code


@pytest.mark.parametrize("change,code", CALLS, ids=str)
def test_call(tcd, change, code):
    assert tcd._linear(layer(tcd), call(tcd, **change), AT, None) == code


# Elements of 2 bytes; x has rows of 64, out and the residual rows of 32, four of each.
OUT = AT + (1 << 16)
OVERLAPS = [
    (dict(out=AT), True),                                              # x itself
    (dict(out=AT, out_stride=64), True),
    (dict(out=AT - 2 * (3 * 32 + 32)), False),                         # up to where x begins
    (dict(out=AT - 2 * (3 * 32 + 31)), True),
    (dict(out=AT + 2 * (3 * 64 + 64)), False),                         # from where x ends
    (dict(out=AT + 2 * (3 * 64 + 63)), True),
    (dict(x_stride=96, out=AT + 2 * 64, out_stride=96), False),        # columns beside x in common rows
    (dict(x_stride=96, out=AT + 2 * 63, out_stride=96), True),
    (dict(x_stride=96, out=AT + 2 * 65, out_stride=96), True),         # (the next row's x)
    (dict(x_stride=96, out=AT - 2 * 32, out_stride=96), False),
    (dict(x_stride=96, out=AT - 2 * 31, out_stride=96), True),
    (dict(x_stride=96, out=AT + 2 * (64 + 96 * 2), out_stride=96), False),
    (dict(x_stride=96, out=AT + 2 * 64, out_stride=192), True),        # (interleaved rows of other strides)
    (dict(n_tokens=1, out=AT + 2 * 64), False),
    (dict(n_tokens=1, out=AT + 2 * 63), True),
    (dict(residual=OUT, residual_stride=32), False),                   # in place
    (dict(residual=OUT, residual_stride=40), True),
    (dict(residual=OUT + 2, residual_stride=32), True),
    (dict(residual=OUT + 2 * 32, out_stride=64, residual_stride=64), False),
    (dict(n_tokens=1, residual=OUT, residual_stride=40), False),
    (dict(residual=AT, residual_stride=32), False),                    # x, which is read as well
]


@pytest.mark.parametrize("change,refused", OVERLAPS, ids=str)
def test_out_overlaps(tcd, change, refused):
    """(Device 63 is not there: what is not refused ends at that.)"""
    w = AT + (1 << 18)
    change = dict(dict(out=OUT), **change)
    code = tcd._linear(layer(tcd, weight=w, device=63), call(tcd, **change), AT, None)
    assert code == (INVALID if refused else CUDA)


@pytest.mark.parametrize("what", ["weight", "gate", "bias", "gate_bias"])
def test_out_overlaps_weights(tcd, what):
    w = dict(weight=AT + (1 << 18), gate=AT + (1 << 19), gate_stride=64, bias=AT + (1 << 17),
             gate_bias=AT + (1 << 17) + 64)
    for at, refused in ((OUT, False), (w[what], True), (w[what] - 2 * 127, True)):
        assert tcd._linear(layer(tcd, device=63, **w), call(tcd, out=at), AT, None) == (INVALID if refused else CUDA)


def test_missing(tcd):
    assert tcd._linear(None, call(tcd), AT, None) == INVALID
    assert tcd._linear(layer(tcd), None, AT, None) == INVALID
    assert tcd._linear(layer(tcd), call(tcd), None, None) == INVALID


def test_no_tokens_is_no_launch(tcd):
    """(x and out may be NULL then.)"""
    assert tcd._linear(layer(tcd), call(tcd, n_tokens=0, x=None, out=None), AT, None) == 0


def test_structures_match_the_header(tcd):
    """Sizes of the C structures on a 64-bit host."""
    assert ctypes.sizeof(tcd._LinearWeights) == 72
    whole = type("Call", (ctypes.Structure,), {"_fields_": [
        (n, ctypes.c_void_p if n in ("x", "residual", "out") else ctypes.c_int32 if n in ("n_tokens", "withhold") else
         ctypes.c_int64) for n in CALL]})
    c = whole.from_buffer_copy(tcd._pack_call(*range(1, 10)) + bytes(8))
    assert [getattr(c, n) for n in CALL] == list(range(1, 10))
