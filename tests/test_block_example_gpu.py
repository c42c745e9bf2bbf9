"""The example block: prompts followed by tokens give what whole prompts give."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    import selective_block
    return selective_block


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_then_tokens_is_the_whole_prompt(example, dtype):
    """Both ways round at the same places (the convolution's and scan's
    outputs, the projections, the norm), so they differ by the order of the
    scan's fp32 sums and, in bf16, by roundings that fall the other way: a
    few half ulps (2^-9) of values whose rows have unit mean square, carried
    through a unit-variance projection of 96 channels."""
    torch.backends.cuda.matmul.allow_tf32 = False
    block = example.SelectiveBlock(64, 96, states=16, dtype=dtype)
    out, state = example.serve(block, [37, 1, 150, 5], 6, 64)
    tol = 2.0 ** -5 if dtype == torch.bfloat16 else 1e-4
    assert out[0] <= tol * out[1], out
    assert state[0] <= tol * state[1], state
