"""Tensors of 16-bit elements that begin in the upper half of a 4-byte word: their
first elements, which single-element copies load apart."""
import pytest
import torch

import gated_deltanet_linear_chunk_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def at_odd(t):
    """The same rows from the second element of a buffer that begins with NaN."""
    buf = torch.full((t.numel() + 1,), float("nan"), dtype=t.dtype, device=t.device)
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


def normal(*shape, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").bfloat16()


@pytest.mark.parametrize("tokens,channels", [(1, 1), (1, 8), (5, 8), (40, 8), (40, 9), (300, 264)])
@pytest.mark.parametrize("width", [2, 4, 8])
def test_conv(tokens, channels, width):
    x, w = normal(tokens, channels), normal(channels, width, seed=1).float()
    cu = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    want, _ = gdn.gdn_short_conv(x, w, cu, activation="silu")
    got, _ = gdn.gdn_short_conv(at_odd(x), w, cu, activation="silu")
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [1, 3, 700])
@pytest.mark.parametrize("dim", [4097, 8192, 9001, 16384])
def test_norm_of_long_rows(rows, dim):
    """Sums of other lanes' words: up to a rounding of the result (2^-8 of it) and
    of its statistic."""
    y, g, r = (normal(rows, dim, seed=s) for s in range(3))
    w = normal(dim, seed=3).float()
    want, want_next = gdn.gdn_norm_gate_residual(y, w, g, r, w)
    for a in ((at_odd(y), g, r), (y, at_odd(g), r), (y, g, at_odd(r)),
              (at_odd(y), at_odd(g), at_odd(r))):
        got, got_next = gdn.gdn_norm_gate_residual(a[0], w, a[1], a[2], w)
        for u, v in ((got, want), (got_next, want_next)):
            assert torch.allclose(u.float(), v.float(), rtol=2.0 ** -7, atol=1e-6)
