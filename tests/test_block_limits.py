"""Sizes past what the block operators' 32-bit indices hold are refused, whatever
the pointers; no launch is made, so no GPU is needed."""
import pytest

import gated_deltanet_linear_chunk_gb300 as gdn
from gated_deltanet_linear_chunk_gb300.block import ConvProblem, SsmProblem

INVALID = 1
A = 0x100000  # an aligned fake device address; never dereferenced here
MOST = (1 << 30) - 1  # sequences and tokens


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return gdn.library()


@pytest.mark.parametrize("seqs", [MOST + 1, (1 << 31) - 1])
def test_more_sequences_than_the_search_holds(lib, seqs):
    """The search of a token's sequence adds two sequence numbers.  (A number
    that 32 bits do not hold reaches the library as their largest.)"""
    p = ConvProblem(seqs, 10, 16, 4, 0, 1, 16, 16)
    assert lib.gdn_short_conv(p, A, A + 4096, None, A + 8192, None, A + 12288, None, None) == INVALID
    p = SsmProblem(seqs, 10, 16, 8, 1, 0, 1, 16, 16, 8, 8, 16, 16, None, 0)
    at = [A + 65536 * i for i in range(5)]
    assert lib.gdn_selective_scan(p, *at, None, None, None, A + (1 << 20), None, A + (2 << 20), None,
                                  None) == INVALID
    assert lib.gdn_selective_scan_workspace_size(p) == 0


def test_more_tokens_than_offsets_hold(lib):
    p = ConvProblem(2, MOST + 1, 16, 4, 0, 1, 16, 16)
    assert lib.gdn_short_conv(p, A, A + 4096, None, A + 8192, None, A + 12288, None, None) == INVALID
