"""The selective scan over its whole accepted range, however its tokens are cut
into windows: growing states, and infinities where the definition has them."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_chunk_gb300 as gdn

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def cu_of(*lens):
    return torch.tensor([0, *lens], device="cuda").cumsum(0).to(torch.int32)


def definition(x, dt, A, B, C, state):
    """Outputs and final state of one sequence, token by token in 64 bits."""
    x, dt, A, B, C, h = (t.double().cpu().numpy() for t in (x, dt, A, B[:, 0], C[:, 0], state[0]))
    out = np.empty_like(x)
    with np.errstate(all="ignore"):
        for t in range(len(x)):
            h = np.exp(dt[t][:, None] * A) * h + (dt[t] * x[t])[:, None] * B[t]
            out[t] = (C[t] * h).sum(1)
    return out, h[None]


# (channels, tokens): windows of 8 tokens joined in one run, of 8 in sixteen
# runs of 40 tokens, and of 22 in four runs of 308.
CUTS = [(64, 24), (64, 640), (2048, 1200)]


def growth(channels, tokens, states=2):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens)

    def positive(*shape):
        return torch.rand(*shape, generator=gen, device="cuda") + 0.5
    A = positive(channels, states)
    B, C = positive(tokens, 1, states), positive(tokens, 1, states)
    return positive(tokens, channels), A, B, C


def check_growth(x, dt, A, B, C, state, live, exponent):
    """All terms are positive, so errors are relative: per token that a value
    grows for (`live`) 8 u of products, sums and the exponential, and u times
    the whole growth's exponent for its steps' products and sums."""
    T = len(x)
    out, fin = gdn.gdn_selective_scan(x, dt, A, B, C, cu_of(T), initial_state=state,
                                      output_final_state=True)
    first = state if state is not None else torch.zeros(1, *A.shape, device="cuda")
    w_out, w_fin = definition(x, dt, A, B, C, first)
    assert np.isfinite(w_out).all() and w_out.max() < 1e38
    rel = (8.0 + exponent) * live * U
    for got, want in ((out, w_out), (fin, w_fin)):
        got = got.double().cpu().numpy()
        assert np.isfinite(got).all(), f"{(~np.isfinite(got)).sum()} of {got.size} not finite"
        assert (np.abs(got - want) <= rel * want + 1e-37).all()


@pytest.mark.parametrize("channels,tokens", CUTS)
@pytest.mark.parametrize("start", [False, True])
def test_growing_states_before_their_first_input(channels, tokens, start):
    """A state that is zero stays zero however much it would have grown: whole
    windows and runs of them multiply it by more than fp32 holds."""
    assert gdn.gdn_selective_scan_workspace_size(1, tokens, channels, 2, 1, torch.float32) > 0
    x, A, B, C = growth(channels, tokens)
    live = 4
    x[:-live] = 0.0
    step = 13.0 if tokens == 24 else 6.0
    dt = torch.full_like(x, step)
    state = torch.zeros(1, channels, 2, device="cuda") if start else None
    check_growth(x, dt, A, B, C, state, live, 1.5 * step * live)


@pytest.mark.parametrize("channels,tokens", CUTS)
def test_tiny_states_that_grow_by_more_than_fp32_holds(channels, tokens):
    """From 1e-30 by e^103 to about 1e15, inside one window or run."""
    x, A, B, C = growth(channels, tokens)
    x.zero_()
    A.fill_(1.0)
    dt = torch.zeros_like(x)
    at, live = tokens // 3, 8  # a window's first token where there are three
    dt[at:at + live] = 103.0 / live
    state = torch.full((1, channels, 2), 1e-30, device="cuda")
    check_growth(x, dt, A, B, C, state, live, 103.0)
