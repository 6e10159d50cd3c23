"""Host bookkeeping of cache pages (tc_pages): against a dictionary model under
random calls, the sharing rules of forks, and every refusal (CPU only)."""
import ctypes
import random

import pytest


def held(pool, seq, width=64):
    return [x for x in pool.row(seq, width).tolist() if x >= 0]


def test_lowest_pages_first_and_back_after_close(tcd):
    p = tcd.PagePool(10, 16)
    a, b = p.open(), p.open()
    assert p.reserve(a, 0, 33) == [] and p.reserve(b, 0, 16) == []
    assert held(p, a) == [0, 1, 2] and held(p, b) == [3] and p.free == 6
    p.close_seq(a)
    assert p.free == 9
    c = p.open()
    assert c == a
    p.reserve(c, 0, 17)
    assert held(p, c) == [0, 1]


def test_fork_shares_until_written(tcd):
    p = tcd.PagePool(10, 16)
    a = p.open()
    p.reserve(a, 0, 40)                       # pages 0 1 2, the last one holds slots 32..39
    b = p.fork(a, 40)
    c = p.fork(a, 32)                         # two full pages
    assert held(p, b) == [0, 1, 2] and held(p, c) == [0, 1] and p.free == 7
    assert p.reserve(b, 40, 41) == [(2, 3)]   # shared and partly filled: a copy
    assert held(p, b) == [0, 1, 3] and held(p, a) == [0, 1, 2]
    assert p.reserve(a, 40, 41) == []         # now its own
    assert p.reserve(c, 32, 50) == [] and held(p, c) == [0, 1, 4, 5]
    assert p.reserve(c, 16, 18) == [] and held(p, c) == [0, 6, 4, 5]   # starts on a page: fresh, no copy
    p.close_seq(a)
    assert held(p, b) == [0, 1, 3]
    p.close_seq(b)
    p.close_seq(c)
    assert p.free == 10


def test_trim(tcd):
    p = tcd.PagePool(8, 16)
    a = p.open()
    p.reserve(a, 0, 100)
    p.trim(a, 33)
    assert held(p, a) == [0, 1, 2] and p.free == 5
    p.trim(a, 1000)
    assert held(p, a) == [0, 1, 2]
    p.trim(a, 0)
    assert held(p, a) == [] and p.free == 8


@pytest.mark.parametrize("seed", range(6))
def test_random_calls_against_a_model(tcd, seed):
    """The model: each sequence's list of pages; a page is free when no list
    has it.  Tables, copies and free counts agree after every call."""
    r = random.Random(seed)
    n, s = r.choice([5, 30, 130]), r.choice([1, 16, 64])
    pool, model = tcd.PagePool(n, s), {}

    def free():
        used = {x for t in model.values() for x in t}
        return [i for i in range(n) if i not in used]

    for _ in range(400):
        op = r.choice(["open", "close", "reserve", "reserve", "reserve", "fork", "trim"])
        seq = r.choice(sorted(model)) if model else None
        if op == "open" or seq is None:
            if len(model) < 12:
                got = pool.open()
                assert got == min(set(range(13)) - set(model))
                model[got] = []
        elif op == "close":
            pool.close_seq(seq)
            del model[seq]
        elif op == "trim":
            at = r.randrange(0, s * 8)
            pool.trim(seq, at)
            model[seq] = model[seq][:-(-at // s)]
        elif op == "fork" and len(model) < 12:
            at = r.randint(0, len(model[seq]) * s)
            child = pool.fork(seq, at)
            model[child] = model[seq][:-(-at // s)]
        elif op == "reserve":
            a = r.randint(0, len(model[seq]) * s)
            b = a + r.randint(0, 3 * s)
            t, fr, copies = list(model[seq]), free(), []
            shared = {x for q, u in model.items() if q != seq for x in u}
            for i in range(a // s, -(-b // s) if b > a else a // s):
                if i < len(t) and t[i] not in shared:
                    continue
                if not fr:
                    t = None
                    break
                if i >= len(t):
                    t.append(fr.pop(0))
                else:
                    new = fr.pop(0)
                    if i == a // s and a % s:
                        copies.append((t[i], new))
                    t[i] = new
            if t is None:
                with pytest.raises(tcd.TcError) as e:
                    pool.reserve(seq, a, b)
                assert e.value.name == "TC_ERR_CAPACITY"
            else:
                assert pool.reserve(seq, a, b) == copies
                model[seq] = t
        for q, t in model.items():
            assert held(pool, q, max(len(t), 1)) == t
        assert pool.free == len(free())


def test_refusals(tcd):
    for pages, size in ((0, 16), (4, 0), (-1, 16)):
        with pytest.raises(tcd.TcError) as e:
            tcd.PagePool(pages, size)
        assert e.value.name == "TC_ERR_INVALID_ARG"
    p = tcd.PagePool(4, 16)
    a = p.open()
    p.reserve(a, 0, 16)
    for bad in (lambda: p.reserve(7, 0, 1), lambda: p.reserve(-1, 0, 1), lambda: p.reserve(a, 17, 18),
                lambda: p.reserve(a, 5, 4), lambda: p.reserve(a, -1, 4), lambda: p.fork(a, 17),
                lambda: p.fork(a, -1), lambda: p.fork(9, 0), lambda: p.trim(a, -1), lambda: p.trim(9, 0),
                lambda: p.close_seq(9), lambda: p.row(9, 4)):
        with pytest.raises(tcd.TcError) as e:
            bad()
        assert e.value.name == "TC_ERR_INVALID_ARG"
    for bad in (lambda: p.reserve(a, 0, 65), lambda: p.reserve(a, 16, 1 << 60), lambda: p.row(a, 0)):
        with pytest.raises(tcd.TcError) as e:
            bad()
        assert e.value.name == "TC_ERR_CAPACITY"
    assert held(p, a) == [0] and p.free == 3
    p.close_seq(a)
    with pytest.raises(tcd.TcError):
        p.close_seq(a)
    null = ctypes.c_void_p()
    assert tcd._pages_create(4, 16, None) == 1
    assert tcd._pages_open(null, None) == 1 and tcd._pages_free_count(null, None) == 1
    tcd._pages_destroy(null)
