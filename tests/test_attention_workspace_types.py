"""The attention's workspace query, without a GPU: no bytes for caches whose type
the call refuses."""
import pytest

import gated_deltanet_linear_chunk_gb300 as gdn
from test_attention_abi import attention_problem, cache


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return gdn.library()


def test_no_workspace_for_types_that_are_refused(lib):
    size = lib.gdn_paged_attention_workspace_size
    for dtype in (0, 1, 2, 3):
        for held in (0, 1, 2, 3, 4):
            fits = (dtype, held) in ((0, 0), (1, 1), (0, 3))
            assert (size(attention_problem(dtype=dtype), cache(dtype=held)) > 0) == fits, (dtype, held)
