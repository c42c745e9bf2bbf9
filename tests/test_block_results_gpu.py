"""Results of the block operators written into columns of a wider tensor, calls
from several host threads, and the convolution before the layer it serves."""
import threading

import numpy as np
import pytest
import torch

import block_ref as ref
import gated_deltanet_linear_chunk_gb300 as gdn

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def maker(seed, dtype=torch.float32):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype=dtype, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)
    return normal


def cu_of(*lens):
    return torch.tensor([0, *lens], device="cuda").cumsum(0).to(torch.int32)


class Columns:
    """[rows, width] as columns of a wider tensor of NaN, from the 16th ("even":
    rows at 16-byte boundaries) or the 3rd ("odd") on."""

    def __init__(self, rows, width, dtype, place):
        lead = 16 if place == "even" else 3
        pad = -(width + lead) % 16 + 16 if place == "even" else 4
        self.whole = torch.full((rows, lead + width + pad), float("nan"), dtype=dtype, device="cuda")
        self.lead, self.width = lead, width
        self.t = self.whole[:, lead:lead + width]

    def untouched(self):
        return (self.whole[:, :self.lead].isnan().all()
                and self.whole[:, self.lead + self.width:].isnan().all())


PLACES = pytest.mark.parametrize("place", ["even", "odd"])
DTYPES = pytest.mark.parametrize("dtype", TYPES)


@PLACES
@DTYPES
@pytest.mark.parametrize("C", [40, 37])
def test_conv_into_columns(place, dtype, C):
    """A channel's sum does not depend on where it is written: the same bits."""
    n = maker(1, TYPES[dtype])
    x, w, b = n(150, C), n(C, 4, dtype=torch.float32), n(C, dtype=torch.float32)
    out = Columns(150, C, TYPES[dtype], place)
    kw = dict(bias=b, activation="silu")
    want, _ = gdn.gdn_short_conv(x, w, cu_of(100, 0, 50), **kw)
    got, _ = gdn.gdn_short_conv(x, w, cu_of(100, 0, 50), out=out.t, **kw)
    assert got is out.t and torch.equal(got, want) and out.untouched()

    state = n(150, 3, C)
    out = Columns(150, C, TYPES[dtype], place)
    want = gdn.gdn_short_conv_step(x, w, state.clone(), **kw)
    got = gdn.gdn_short_conv_step(x, w, state, out=out.t, **kw)
    assert torch.equal(got, want) and out.untouched()


@PLACES
@DTYPES
@pytest.mark.parametrize("d,S,G", [(40, 16, 1), (37, 5, 1), (48, 16, 3)])
def test_scan_into_columns(place, dtype, d, S, G):
    n, f32, T = maker(2, TYPES[dtype]), torch.float32, 300
    x, dt, z, B, C = n(T, d), n(T, d), n(T, d), n(T, G, S), n(T, G, S)
    A, D, b = -n(d, S, dtype=f32).abs(), n(d, dtype=f32), n(d, dtype=f32)
    kw = dict(D=D, z=z, dt_bias=b, dt_softplus=True)
    for lens in ((T,), (100, 0, 150, 50)):
        out = Columns(T, d, TYPES[dtype], place)
        want, _ = gdn.gdn_selective_scan(x, dt, A, B, C, cu_of(*lens), **kw)
        got, _ = gdn.gdn_selective_scan(x, dt, A, B, C, cu_of(*lens), out=out.t, **kw)
        assert torch.equal(got, want) and out.untouched()

    state = n(T, d, S, dtype=f32)
    out = Columns(T, d, TYPES[dtype], place)
    want = gdn.gdn_selective_scan_step(x, dt, A, B, C, state.clone(), **kw)
    got = gdn.gdn_selective_scan_step(x, dt, A, B, C, state, out=out.t, **kw)
    assert torch.equal(got, want) and out.untouched()


@PLACES
@pytest.mark.parametrize("types", ["bf16-bf16", "bf16-f32", "f32-f32"])
@pytest.mark.parametrize("rows,dim", [(7, 64), (7, 37), (300, 1040), (700, 8200), (700, 4100),
                                      (400, 9001)])
def test_norm_into_columns(place, types, rows, dim):
    """Another alignment may take other words and so sum the squares in another
    order: against 64 bits, within the bounds derived for them."""
    dt, rt = (TYPES[k] for k in types.split("-"))
    n = maker(3, dt)
    y, g, r = n(rows, dim), n(rows, dim), n(rows, dim, dtype=rt)
    w, v = n(dim, dtype=torch.float32), n(dim, dtype=torch.float32)
    out, nxt = Columns(rows, dim, rt, place), Columns(rows, dim, dt, place)
    got, got_next = gdn.gdn_norm_gate_residual(y, w, g, r, v, out=out.t, next_out=nxt.t)
    assert got is out.t and got_next is nxt.t and out.untouched() and nxt.untouched()
    u = {torch.bfloat16: ref.U_BF16, torch.float32: 2 * ref.U}
    wide = [t.double().cpu().numpy() for t in (y, w, g, r, v)]
    want, bound, want_next, bound_next = ref.norm(*wide, u_out=u[rt], u_next=u[dt])
    assert (np.abs(got.double().cpu().numpy() - want) <= bound + 1e-30).all()
    assert (np.abs(got_next.double().cpu().numpy() - want_next) <= bound_next + 1e-30).all()


def test_calls_from_host_threads():
    """Each thread on its own stream: the same bits as one call after another."""
    threads, repeats, T, d = 4, 8, 500, 96
    one = torch.ones(d, device="cuda")

    def problem(i):
        n = maker(10 + i, torch.bfloat16)
        return dict(x=n(T, d), w=n(d, 4, dtype=torch.float32), dt=n(T, d), B=n(T, 1, 13), C=n(T, 1, 13),
                    A=-n(d, 13, dtype=torch.float32).abs(), s=n(9, 3, d), h=n(9, d, 13, dtype=torch.float32))

    def calls(p):
        c, w = gdn.gdn_short_conv(p["x"], p["w"], cu_of(T), activation="silu", output_final_state=True)
        y, h = gdn.gdn_selective_scan(c, p["dt"], p["A"], p["B"], p["C"], cu_of(T), dt_softplus=True,
                                      output_final_state=True)
        m, k = gdn.gdn_norm_gate_residual(y, one, gate=c, residual=p["x"], next_weight=one)
        t = gdn.gdn_short_conv_step(p["x"][:9], p["w"], p["s"], new_state=torch.empty_like(p["s"]))
        u = gdn.gdn_selective_scan_step(t, p["dt"][:9], p["A"], p["B"][:9], p["C"][:9], p["h"],
                                        new_state=torch.empty_like(p["h"]), dt_softplus=True)
        return [c, w, y, h, m, k, t, u]
    problems = [problem(i) for i in range(threads)]
    want = [calls(p) for p in problems]
    torch.cuda.synchronize()
    got, errors = [[] for _ in range(threads)], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(repeats):
                    got[i].append(calls(problems[i]))
            stream.synchronize()
        except BaseException as e:  # reported on the main thread
            errors.append(e)
    running = [threading.Thread(target=work, args=(i,)) for i in range(threads)]
    for t in running:
        t.start()
    for t in running:
        t.join()
    assert not errors, errors
    for i in range(threads):
        assert len(got[i]) == repeats
        for results in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(results, want[i]))


def test_convolution_before_the_layer():
    """q, k and v of one projection, convolved slice by slice: each result is
    contiguous, as the layer's prefill takes it, and has the bits of the whole
    projection's convolution.  Then the gated norm of every value head."""
    lens, Hk, Hv, d = [300, 1, 150], 2, 6, 128
    T, widths = sum(lens), [Hk * d, Hk * d, Hv * d]
    n = maker(4, torch.bfloat16)
    proj, gates = n(T, sum(widths) + Hv * d), (n(T, Hv, dtype=torch.float32) for _ in range(2))
    w, cu = n(sum(widths), 4, dtype=torch.float32, std=0.5), cu_of(*lens)
    window = n(len(lens), 3, sum(widths))
    whole, last = gdn.gdn_short_conv(proj[:, :sum(widths)], w, cu, initial_state=window,
                                     activation="silu", output_final_state=True)
    parts, lasts, at = [], [], 0
    for width in widths:
        cols = slice(at, at + width)
        y, s = gdn.gdn_short_conv(proj[:, cols], w[cols], cu, activation="silu",
                                  initial_state=window[:, :, cols].contiguous(),
                                  output_final_state=True)
        parts.append(y)
        lasts.append(s)
        at += width
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(torch.cat(lasts, 2), last)

    def unit(x):
        x = x.view(T, Hk, d)
        return torch.nn.functional.normalize(x.float(), dim=-1).to(x.dtype)
    g, beta = (torch.sigmoid(t) for t in gates)
    out, _ = gdn.gdn_chunk_prefill(unit(parts[0]), unit(parts[1]), parts[2].view(T, Hv, d), -g, beta,
                                   cu)
    assert out.is_contiguous() and out.isfinite().all()
    gate = proj[:, sum(widths):].reshape(T * Hv, d)
    one = torch.ones(d, device="cuda")
    heads, _ = gdn.gdn_norm_gate_residual(out.view(T * Hv, d), one, gate=gate)
    o = out.view(T * Hv, d).double()
    want = o / torch.sqrt((o * o).mean(1, keepdim=True) + 1e-6)
    want = want * torch.nn.functional.silu(gate.double())
    assert torch.allclose(heads.double(), want, rtol=2.0 ** -7, atol=1e-6)
