"""The norm in place on one row: its strides do not matter."""
import pytest
import torch

import gated_deltanet_linear_chunk_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("over,next_over", [("y", "gate"), ("residual", "y"), ("residual", "gate")])
def test_norm_of_one_row_in_place_under_another_stride(over, next_over):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    wide = {k: torch.randn(3, 200, generator=gen, device="cuda").bfloat16()
            for k in ("y", "gate", "residual")}
    w = torch.randn(128, generator=gen, device="cuda")
    rows = {k: v[1:2, :128] for k, v in wide.items()}      # stride 200
    again = {k: v[1, :128][None] for k, v in wide.items()}  # the same row, stride 128
    assert rows["y"].stride(0) != again["y"].stride(0)
    want, want_next = gdn.gdn_norm_gate_residual(**rows, weight=w, next_weight=w)
    out, nxt = gdn.gdn_norm_gate_residual(**rows, weight=w, next_weight=w, out=again[over],
                                          next_out=again[next_over])
    assert torch.equal(out, want) and torch.equal(nxt, want_next)
    assert torch.equal(wide[over][1, :128], want[0])
    assert torch.equal(wide[next_over][1, :128], want_next[0])
