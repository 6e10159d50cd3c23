"""Which buffers the cache object gives to calls without their own (CPU: the
capture queries and the device memory are stand-ins)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def world(tcd, monkeypatch):
    """Captures by stream handle, watched words by capture, and a cache on them."""
    captures, words, made = {}, {}, []

    def capture_id(stream, ref):
        ref._obj.value = captures.get(stream, 0)
        return 0

    def watch(stream, ref):
        word = words.setdefault(captures[stream], ctypes.c_int32(0))
        ref._obj.contents = word
        return 0

    def empty(n, dtype, device, stream, zero=False):
        assert not captures.get(stream), "memory of a stream that is being captured would be the graph's own"
        made.append(stream)
        return torch.zeros(n, dtype=dtype)

    monkeypatch.setattr(tcd, "_capture_id", capture_id)
    monkeypatch.setattr(tcd, "_capture_watch", watch)
    monkeypatch.setattr(tcd, "_capture_unwatch", lambda word: None)
    monkeypatch.setattr(tcd, "_clear_now", lambda p, n, s: 0)
    monkeypatch.setattr(tcd, "_capture_mode", lambda ref: 0)
    monkeypatch.setattr(tcd, "_empty", empty)
    monkeypatch.setattr(tcd, "_stream_aside", lambda device: 900)
    monkeypatch.setattr(tcd, "_held", [])

    def cache():
        c = tcd.KvCache.__new__(tcd.KvCache)
        c.device, c._i32, c._u8, c.workspace_bytes = torch.device("cpu"), torch.int32, torch.uint8, 64
        c._own, c._captured, c._graph_codes = {}, {}, None
        c._capture = ctypes.c_uint64()
        c._capture_ref = ctypes.byref(c._capture)
        c._kvp_keep = None
        return c

    return tcd, captures, words, cache


def test_each_capture_has_a_workspace_of_its_own(world):
    """Two graphs captured one after the other on one stream, two streams of one capture, and calls outside."""
    tcd, captures, words, make = world
    c = make()
    outside = c._workspace(None, 5)
    captures[5] = 1
    first = c._workspace(None, 5)
    captures[6] = 1                                   # (a branch of the same capture)
    branch = c._workspace(None, 6)
    assert c._workspace(None, 5) == first and c._workspace(None, 6) == branch
    captures[5] = 2
    del captures[6]
    second = c._workspace(None, 5)
    del captures[5]
    assert c._workspace(None, 5) == outside
    assert len({x[0] for x in (outside, first, branch, second)}) == 4


def test_buffers_stay_while_the_graph_does(world):
    tcd, captures, words, make = world
    c = make()
    captures[5] = 1
    c._workspace(None, 5)
    (own,) = tcd._held
    del c
    assert tcd._held == [own] and not own.idle()
    words[1].value = 1
    assert own.idle()
    captures[5] = 2
    make()._workspace(None, 5)
    assert len(tcd._held) == 1 and tcd._held[0] is not own


def test_codes_of_captured_calls_are_common_and_not_lost_with_their_graph(world):
    tcd, captures, words, make = world
    c = make()
    captures[5] = 1
    a = c._codes(None, 3, 5)
    words[1].value = 1
    captures[5] = 2
    assert c._codes(None, 7, 5) == a and c._graph_codes.used == [7, 0]
    assert len(c._captured) == 1
    del captures[5]
    assert c._codes(None, 3, 5) != a


def test_a_given_workspace_is_taken(world):
    tcd, captures, words, make = world
    c = make()
    t = torch.zeros(100, dtype=torch.int32)
    assert c._workspace(t, 5) == (t.data_ptr(), 400) and not c._own
    with pytest.raises(ValueError):
        c._workspace(t[::2], 5)
    with pytest.raises(ValueError):
        c._workspace(torch.empty(100, device="meta"), 5)
