"""Results of the prompts' forms that lie over what other blocks of the same call
still read or write are refused, as the steps refuse them; no launch is made."""
import pytest

import gated_deltanet_linear_chunk_gb300 as gdn
from gated_deltanet_linear_chunk_gb300.block import ConvProblem, SsmProblem

INVALID = 1
A = 0x100000  # an aligned fake device address; never dereferenced here


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return gdn.library()


@pytest.mark.parametrize("kw", [dict(out="init"), dict(out="fin"), dict(fin="x"),
                                dict(out="both"), dict(out="x")])
def test_conv(lib, kw):
    at = dict(x=A, w=A + 4096, cu=A + 8192, init=A + 12288, out=A + 16384, fin=A + 20480)
    if kw == dict(out="both"):
        at["out"] = at["fin"] = at["init"]
    else:
        (name, other), = kw.items()
        at[name] = at[other]
    p = ConvProblem(2, 10, 16, 4, 1, 1, 16, 16)
    assert lib.gdn_short_conv(p, at["x"], at["w"], None, at["cu"], at["init"], at["out"], at["fin"],
                              None) == INVALID


@pytest.mark.parametrize("name,other", [("out", "init"), ("out", "fin")] +
                         [("fin", k) for k in ("x", "dt", "a", "b", "c", "z")])
def test_scan(lib, name, other):
    names = ("x", "dt", "a", "b", "c", "skip", "z", "bias", "cu", "init", "out", "fin")
    at = {k: A + 65536 * i for i, k in enumerate(names)}
    at[name] = at[other]
    p = SsmProblem(2, 10, 16, 8, 1, 1, 1, 16, 16, 8, 8, 16, 16, None, 0)
    assert lib.gdn_selective_scan(p, *[at[k] for k in names], None) == INVALID
