"""The example that runs the cache's operators together with the constrained
step: drafting branches of the catalog gives the plain decode's tokens in fewer
forward passes, and every output is in the catalog's language."""
import os
import sys

import pytest

from conftest import ROOT
from gpu_common import torch_mod
from trie_constrained_decoding_gb300 import inputs as I

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_drafted_decode_equals_plain_decode(tcd):
    torch_mod()
    import tree_decode
    plain, steps = tree_decode.decode(tcd, 1)
    drafted, rounds = tree_decode.decode(tcd, 16)
    w = I.tiny()
    names = {tuple(s) for s in w.catalog}
    for t in drafted:
        assert t[-1] == w.stop_id
        parts, cur = [], []
        for x in t[:-1]:
            if x == w.sep_id:
                parts.append(tuple(cur))
                cur = []
            else:
                cur.append(x)
        parts.append(tuple(cur))
        assert len(parts) == 3 and len(set(parts)) == 3 and set(parts) <= names
    assert drafted == plain
    assert rounds < steps
