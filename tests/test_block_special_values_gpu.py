"""Infinities in the selective scan's inputs: results are infinite where the
definition's are, whatever the state count is padded to and with or without
the optional terms."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_chunk_gb300 as gdn

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def definition(a, D, z, state):
    """Outputs and final state of one sequence, token by token in 64 bits."""
    x, dt, A, B, C = (a[k].double().cpu().numpy() for k in ("x", "dt", "A", "B", "C"))
    h = state[0].double().cpu().numpy()
    out = np.empty_like(x)
    with np.errstate(all="ignore"):
        for t in range(len(x)):
            h = np.exp(dt[t][:, None] * A) * h + (dt[t] * x[t])[:, None] * B[t]
            out[t] = (C[t] * h).sum(1)
            if D is not None:
                out[t] += D.double().cpu().numpy() * x[t]
            if z is not None:
                g = z[t].double().cpu().numpy()
                out[t] *= g / (1.0 + np.exp(-g))
    return out, h[None]


def inputs(rows, d, S, dtype, step, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def positive(*shape):
        return torch.rand(*shape, generator=gen, device="cuda") + 0.5
    return dict(x=positive(rows, d).to(dtype), dt=torch.full((rows, d), step, dtype=dtype, device="cuda"),
                A=-positive(d, S), B=positive(rows, 1, S).to(dtype), C=positive(rows, 1, S).to(dtype),
                z=positive(rows, d).to(dtype), D=positive(d), state=positive(1, d, S))


def same_kind(got, want, clean, hit):
    """NaN and infinities where the definition has them, every other channel
    as it is without them."""
    got, clean = got.double().cpu().numpy(), clean.double().cpu().numpy()
    special = ~np.isfinite(want)
    assert special.any()
    assert (np.isnan(got) == np.isnan(want)).all(), "NaN"
    assert (np.isinf(got) == np.isinf(want)).all(), "infinities"
    assert (got[np.isinf(want)] == want[np.isinf(want)]).all(), "signs"
    other = [c for c in range(got.shape[1]) if c not in hit]
    assert np.array_equal(got[:, other], clean[:, other])


# Windows: one, or of ten tokens; what a window's decay leaves of a state is
# less than fp32 holds with the steps of 12.
@pytest.mark.parametrize("rows,step", [(20, 0.125), (300, 0.125), (300, 12.0)])
@pytest.mark.parametrize("S", [1, 3, 4, 13, 16, 33])
@pytest.mark.parametrize("d", [40, 37])
@pytest.mark.parametrize("dtype", TYPES)
def test_scan_infinite_inputs(rows, step, S, d, dtype):
    a = inputs(rows, d, S, TYPES[dtype], step)
    cu = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    hit = (0, 11, d - 1)
    for D, z in ((None, None), (a["D"], None), (None, a["z"])):
        def run(a):
            return gdn.gdn_selective_scan(a["x"], a["dt"], a["A"], a["B"], a["C"], cu, D=D, z=z,
                                          initial_state=a["state"], output_final_state=True)
        clean = run(a)
        b = dict(a, x=a["x"].clone(), dt=a["dt"].clone())
        b["x"][5, 0] = float("inf")
        b["x"][rows - 3, 11] = -float("inf")
        b["dt"][6, d - 1] = float("inf")
        for got, want, base in zip(run(b), definition(b, D, z, b["state"]), clean):
            same_kind(got, want, base, hit)


@pytest.mark.parametrize("S", [1, 3, 16])
@pytest.mark.parametrize("dtype", TYPES)
def test_scan_step_infinite_inputs(S, dtype):
    d = 40
    a = inputs(1, d, S, TYPES[dtype], 0.125)
    for D, z in ((None, None), (a["D"], None), (None, a["z"])):
        def run(a):
            new = torch.empty_like(a["state"])
            out = gdn.gdn_selective_scan_step(a["x"], a["dt"], a["A"], a["B"], a["C"], a["state"],
                                              D=D, z=z, new_state=new)
            return out, new
        clean = run(a)
        b = dict(a, x=a["x"].clone(), dt=a["dt"].clone())
        b["x"][0, 0], b["x"][0, 11], b["dt"][0, d - 1] = float("inf"), -float("inf"), float("inf")
        for got, want, base in zip(run(b), definition(b, D, z, b["state"]), clean):
            same_kind(got, want, base, (0, 11, d - 1))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("S", [3, 16])
@pytest.mark.parametrize("d", [40, 37])
def test_scan_infinite_inputs_among_sequences(in_place, S, d):
    """Sequences that begin, end or go on in a window after one with infinities,
    their final states over the initial ones or apart."""
    lens = [7, 30, 3, 0, 2, 60, 1]
    rows, cuts = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    a = inputs(rows, d, S, torch.bfloat16, 0.125)
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    state = a["state"].repeat(len(lens), 1, 1)

    def run(x):
        fin = state.clone() if in_place else torch.full_like(state, float("nan"))
        out, _ = gdn.gdn_selective_scan(x, a["dt"], a["A"], a["B"], a["C"], cu, z=a["z"],
                                        initial_state=fin if in_place else state, final_state=fin)
        return out, fin
    clean = run(a["x"])
    x = a["x"].clone()
    x[9, 0], x[20, 5], x[38, 5], x[50, d - 1] = float("inf"), -float("inf"), float("inf"), float("inf")
    out, fin = run(x)
    for n, (b, e) in enumerate(zip(cuts[:-1], cuts[1:])):
        one = {k: (v[b:e] if k in ("x", "dt", "B", "C", "z") else v) for k, v in dict(a, x=x).items()}
        w_out, w_fin = definition(one, None, one["z"], state[n:n + 1])
        if np.isfinite(w_out).all():
            assert torch.equal(out[b:e], clean[0][b:e]) and torch.equal(fin[n], clean[1][n])
        else:
            same_kind(out[b:e], w_out, clean[0][b:e], (0, 5, d - 1))
            same_kind(fin[n:n + 1], w_fin, clean[1][n:n + 1], (0, 5, d - 1))
