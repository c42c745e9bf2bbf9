"""The block operators past 32-bit element offsets, over many windows, on
given streams and in captured graphs."""
import pytest
import torch

import gated_deltanet_linear_chunk_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def cu_of(*lens):
    return torch.tensor([0, *lens], device="cuda").cumsum(0).to(torch.int32)


ROWS, WIDTH = 270_000, 8192  # 2.2e9 elements: offsets pass 2^31


def test_conv_and_norm_past_32_bit_offsets():
    """The last rows of a tensor of 2.2e9 elements are those of a small call
    on them."""
    x = torch.empty(ROWS, WIDTH, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.randn(WIDTH, 4, device="cuda")
    out, _ = gdn.gdn_short_conv(x, w, cu_of(ROWS), activation="silu")
    tail = slice(ROWS - 100, ROWS)
    want, _ = gdn.gdn_short_conv(x[tail].clone(), w, cu_of(100), activation="silu",
                                 initial_state=x[None, ROWS - 103:ROWS - 100].clone())
    assert torch.equal(out[tail], want)
    one = torch.randn(WIDTH, device="cuda")
    got, _ = gdn.gdn_norm_gate_residual(x, one, out=out)
    want, _ = gdn.gdn_norm_gate_residual(x[tail].clone(), one)
    assert torch.equal(got[tail], want)


def test_scan_past_32_bit_offsets():
    """Two sequences, the second one past 2^31 elements: it is the same call on
    that sequence alone."""
    first, second = ROWS - 1000, 1000
    x = torch.empty(ROWS, WIDTH, dtype=torch.bfloat16, device="cuda").normal_()
    dt = torch.full((ROWS, 1), -3.0, dtype=torch.bfloat16, device="cuda").expand(ROWS, WIDTH)
    dt = dt.contiguous()
    A = -torch.rand(WIDTH, 4, device="cuda") - 0.5
    B = torch.randn(ROWS, 1, 4, device="cuda").bfloat16()
    out, fin = gdn.gdn_selective_scan(x, dt, A, B, B, cu_of(first, second), z=x, dt_softplus=True,
                                      output_final_state=True)
    tail = slice(first, ROWS)
    want, last = gdn.gdn_selective_scan(x[tail].clone(), dt[tail].clone(), A, B[tail].clone(),
                                        B[tail].clone(), cu_of(second), z=x[tail].clone(),
                                        dt_softplus=True, output_final_state=True)
    # Other windows, another order of the fp32 sums: 2^-8 is one rounding of
    # the result the other way.
    assert (out[tail].float() - want.float()).abs().max() <= 2.0 ** -8 * want.float().abs().max()
    assert (fin[1] - last[0]).abs().max() <= 1e-5 * last.abs().max()


def test_states_past_32_bit_offsets():
    """Steps of so many sequences that the states pass 2^31 elements."""
    n, d, s = 140_000, 1024, 16
    state = torch.full((n, d, s), 0.5, device="cuda")
    x = torch.randn(n, d, device="cuda").bfloat16()
    A = -torch.rand(d, s, device="cuda")
    B = torch.randn(n, 1, s, device="cuda").bfloat16()
    tail = slice(n - 3, n)
    want_state = state[tail].clone()
    want = gdn.gdn_selective_scan_step(x[tail].clone(), x[tail].clone(), A, B[tail].clone(),
                                       B[tail].clone(), want_state, dt_softplus=True)
    out = gdn.gdn_selective_scan_step(x, x, A, B, B, state, dt_softplus=True)
    assert torch.equal(out[tail], want) and torch.equal(state[tail], want_state)


@pytest.mark.parametrize("channels,groups", [(24, 1), (24, 4), (257, 1)])
def test_scan_over_many_windows(channels, groups):
    """Thousands of tokens in hundreds of windows, against the same sequence in
    calls of one window each (under 24 tokens: their states are carried by
    the caller)."""
    T, S = 3000, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    x, dt = normal(T, channels), normal(T, channels) - 3.0
    A = -torch.rand(channels, S, generator=gen, device="cuda") * 4 - 0.1
    B, C = normal(T, groups, S), normal(T, groups, S)
    state = normal(1, channels, S)
    assert gdn.gdn_selective_scan_workspace_size(1, T, channels, S, groups, torch.float32) > 0
    assert gdn.gdn_selective_scan_workspace_size(1, 20, channels, S, groups, torch.float32) == 0
    out, fin = gdn.gdn_selective_scan(x, dt, A, B, C, cu_of(T), dt_softplus=True,
                                      initial_state=state, output_final_state=True)
    want = []
    for t in range(0, T, 20):
        at = slice(t, t + 20)
        y, state = gdn.gdn_selective_scan(x[at], dt[at], A, B[at], C[at], cu_of(20),
                                          dt_softplus=True, initial_state=state,
                                          output_final_state=True)
        want.append(y)
    want = torch.cat(want)
    # fp32 sums in another order: some tens of ulps (2^-24) of the largest.
    assert (out - want).abs().max() <= 1e-5 * want.abs().max()
    assert (fin - state).abs().max() <= 1e-5 * state.abs().max()


def test_given_stream_and_graph_capture():
    """A call given a stream runs there and its results belong to it; a
    captured call replays on new inputs."""
    side = torch.cuda.Stream()
    x = torch.randn(300, 64, device="cuda").bfloat16()
    w = torch.randn(64, 4, device="cuda")
    A = -torch.rand(64, 8, device="cuda")
    B = torch.randn(300, 1, 8, device="cuda").bfloat16()
    one, cu = torch.ones(64, device="cuda"), cu_of(300)
    state = torch.randn(300, 3, 64, device="cuda").bfloat16()
    ssm = torch.randn(300, 64, 8, device="cuda")

    def calls(x, **kw):
        c, _ = gdn.gdn_short_conv(x, w, cu, activation="silu", **kw)
        s, f = gdn.gdn_selective_scan(c, x, A, B, B, cu, z=x, dt_softplus=True,
                                      output_final_state=True, **kw)
        n, m = gdn.gdn_norm_gate_residual(s, one, gate=x, residual=c, next_weight=one, **kw)
        t = gdn.gdn_short_conv_step(x, w, state, new_state=torch.empty_like(state), **kw)
        u = gdn.gdn_selective_scan_step(t, x, A, B, B, ssm, new_state=torch.empty_like(ssm),
                                        dt_softplus=True, **kw)
        return [c, s, f, n, m, t, u]
    want = calls(x)
    torch.cuda.synchronize()
    late = torch.empty_like(x)
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)
        late.copy_(x)
    got = calls(late, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    graph, static = torch.cuda.CUDAGraph(), torch.zeros_like(x)
    with torch.cuda.graph(graph):
        got = calls(static)
    static.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_of_the_binding():
    """Tensors that the checks must not let through, on the device."""
    x = torch.randn(6, 16, device="cuda")
    w = torch.randn(16, 4, device="cuda")
    cu = cu_of(6)
    A, B = -torch.rand(16, 8, device="cuda"), torch.randn(6, 1, 8, device="cuda")
    bad = ValueError
    with pytest.raises(bad):  # a slice of columns as a parameter
        gdn.gdn_short_conv(x, torch.randn(16, 8, device="cuda")[:, :4], cu)
    with pytest.raises(bad):  # overlapping rows as the result
        gdn.gdn_short_conv(x, w, cu, out=torch.empty(1, 16, device="cuda").expand(6, 16))
    with pytest.raises(bad):  # a state of another width
        gdn.gdn_short_conv(x, w, cu, initial_state=torch.zeros(1, 2, 16, device="cuda"))
    with pytest.raises(bad):  # lengths on the host
        gdn.gdn_short_conv(x, w, cu.cpu())
    with pytest.raises(TypeError):
        gdn.gdn_short_conv(x, w, cu.long())
    with pytest.raises(bad):  # B's states not contiguous
        gdn.gdn_selective_scan(x, x, A, torch.randn(6, 8, 1, device="cuda").transpose(1, 2)
                               .expand(6, 2, 8), B, cu)
    with pytest.raises(TypeError):
        gdn.gdn_selective_scan(x, x.bfloat16(), A, B, B, cu)
    with pytest.raises(bad):
        gdn.gdn_selective_scan(x, x, A[:, :7], B, B, cu)
    with pytest.raises(gdn.GDNError):  # more states than supported
        gdn.gdn_selective_scan(x, x, -torch.rand(16, 65, device="cuda"),
                               torch.randn(6, 1, 65, device="cuda"),
                               torch.randn(6, 1, 65, device="cuda"), cu)
    with pytest.raises(gdn.GDNError):  # three groups of sixteen channels
        B3 = torch.randn(6, 3, 8, device="cuda")
        gdn.gdn_selective_scan(x, x, A, B3, B3, cu)
    with pytest.raises(gdn.GDNError):  # too small a workspace
        y = torch.randn(600, 16, device="cuda")
        B6 = torch.randn(600, 1, 8, device="cuda")
        gdn.gdn_selective_scan(y, y, A, B6, B6, cu_of(600),
                               workspace=torch.empty(16, device="cuda"))
    with pytest.raises(gdn.GDNError):  # the result over an input
        gdn.gdn_short_conv(x, w, cu, out=x)
    with pytest.raises(bad):
        gdn.gdn_norm_gate_residual(x, next_out=x)
    with pytest.raises(gdn.GDNError):
        gdn.gdn_norm_gate_residual(x, eps=-1.0)


@pytest.mark.parametrize("states", [16, 13, 64])
def test_scan_step_of_many_pairs(states):
    """More (channel tile, sequence) pairs than blocks, so that a block passes
    from one tile to the next: the same bits as the sequences in small
    batches, in place and apart."""
    n, d, groups = 900, 700, 2
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)
    x, dt, z = normal(n, d), normal(n, d), normal(n, d)
    B, C = normal(n, groups, states), normal(n, groups, states)
    A = -torch.rand(d, states, generator=gen, device="cuda") * 4
    D, bias = normal(d, dtype=torch.float32), normal(d, dtype=torch.float32)
    state = normal(n, d, states, dtype=torch.float32)
    kw = dict(D=D, dt_bias=bias, dt_softplus=True)
    want, want_state = [], []
    for i in range(0, n, 60):
        at = slice(i, i + 60)
        s = state[at].clone()
        want.append(gdn.gdn_selective_scan_step(x[at], dt[at], A, B[at], C[at], s, z=z[at], **kw))
        want_state.append(s)
    new = torch.empty_like(state)
    out = gdn.gdn_selective_scan_step(x, dt, A, B, C, state, z=z, new_state=new, **kw)
    assert torch.equal(out, torch.cat(want)) and torch.equal(new, torch.cat(want_state))
    out = gdn.gdn_selective_scan_step(x, dt, A, B, C, state, z=z, **kw)
    assert torch.equal(out, torch.cat(want)) and torch.equal(state, torch.cat(want_state))
