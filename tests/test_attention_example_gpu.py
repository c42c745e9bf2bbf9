"""The example attention block: prompts followed by tokens give what whole
prompts give."""
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
    import attention_block
    return attention_block


@pytest.mark.parametrize("drafted", [1, 3, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_then_tokens_is_the_whole_prompt(example, dtype, drafted):
    """Both ways attend over the same keys and values, by other kernels: they
    differ by the weights' and outputs' roundings (2^-8 each in bf16) and by the
    gate's, carried through a unit-variance projection of 768 elements whose
    differences are independent: some 2^-7 of values of unit mean square, the
    largest of the differences a few times that."""
    torch.backends.cuda.matmul.allow_tf32 = False
    block = example.AttentionBlock(64, dtype=dtype)
    off, most = example.serve(block, [37, 1, 150, 5], 24 // drafted, drafted, 64)
    tol = 2.0 ** -5 if dtype == torch.bfloat16 else 1e-4
    assert off <= tol * most, (off, most)
