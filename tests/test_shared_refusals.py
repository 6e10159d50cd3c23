"""tc_attend_shared's checks of its arguments (CPU: a refused call touches no device)."""
import ctypes

import pytest

from test_cache_buffers import world  # noqa: F401  (a fixture)

INVALID, CAPACITY, UNSUPPORTED = 1, 10, 11
AT = 1 << 20   # (an address that is never read)


def arguments(tcd, **kw):
    v = dict(layer=0, batch=4, n_tokens=4, groups=1, cu_seqs=AT, shared_lens=AT, q_heads=8, kv_heads=2, page=16, words=0,
             tree=None, max_tokens=1)
    v.update(kw)
    kv = tcd._Kv(AT, 0, 0, 1, 8, v["kv_heads"], v["page"], 64, 0)
    t = tcd._Tokens(v["batch"], v["n_tokens"], AT, AT, AT, 4)
    a = tcd._Attend(AT, 512, v["q_heads"], v["max_tokens"], 1.0, v["tree"], v["words"], AT, 512, None, 0, 0)
    return kv, v["layer"], t, a, tcd._Shared(v["groups"], v["cu_seqs"], v["shared_lens"]), AT, 1 << 40, AT, None


@pytest.mark.parametrize("change,code", [
    (dict(groups=0), INVALID), (dict(groups=-1), INVALID), (dict(groups=5), INVALID), (dict(cu_seqs=None), INVALID),
    (dict(shared_lens=None), INVALID), (dict(layer=1), INVALID), (dict(batch=0), INVALID), (dict(page=24), UNSUPPORTED),
    (dict(q_heads=7), UNSUPPORTED), (dict(batch=65537), CAPACITY), (dict(max_tokens=-1), INVALID),
    (dict(tree=AT, words=1, max_tokens=65), CAPACITY), (dict(tree=AT, words=5), CAPACITY),
], ids=str)
def test_arguments(tcd, change, code):
    assert tcd._attend_shared(*arguments(tcd, **change)) == code


def test_missing(tcd):
    a = list(arguments(tcd))
    for i, code in ((0, INVALID), (2, INVALID), (3, INVALID), (4, INVALID), (7, INVALID)):
        b = list(a)
        b[i] = None
        assert tcd._attend_shared(*b) == code
    n = ctypes.c_int64()
    assert tcd._attend_shared_workspace(None, 4, 8, ctypes.byref(n)) == INVALID


def test_workspaces_that_are_outgrown(world):  # noqa: F811
    """A larger one takes a smaller one's place; a captured call's stays, as its graph uses it."""
    tcd, captures, words, make = world
    c = make()
    assert c._workspace(None, 5)[1] == 64
    more = c._workspace(None, 5, need=100)
    assert more[1] == 100 and c._workspace(None, 5) == more and c._workspace(None, 5, need=99) == more
    captures[5] = 1
    first = c._workspace(None, 5)
    second = c._workspace(None, 5, need=200)
    assert first[1] == 64 and second[1] == 200 and c._workspace(None, 5) == second
    assert [t.data_ptr() for t in c._captured[1, 5].outgrown] == [first[0]]
