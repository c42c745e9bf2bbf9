"""The block operators (short convolution, selective scan, block norm) against
plain 64-bit references, element by element within derived bounds."""
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


def u_of(dtype):
    return ref.U_BF16 if dtype == torch.bfloat16 else 2 * ref.U


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, want, bound, what):
    """Every element within its bound (and finite where the reference is)."""
    got = f64(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound + 1e-30)
    if bad.any():
        i = tuple(int(k[0]) for k in np.nonzero(bad))
        pytest.fail(f"{what}: {bad.sum()} of {bad.size} outside, first at {i}: {got[i]!r}, "
                    f"reference {want[i]!r}, bound {bound[i]:.3g}")


class Draw:
    def __init__(self, seed):
        self.rng = np.random.default_rng(seed)

    def __call__(self, *shape, dtype=torch.float32, std=1.0, mean=0.0):
        v = self.rng.standard_normal(shape) * std + mean
        return torch.from_numpy(v).to(dtype).cuda()

    def rows(self, n, width, dtype, wide):
        """[n, width]; wide: a slice of the columns of a larger tensor, 16-byte
        aligned ("even") or not ("odd")."""
        if not wide:
            return self(n, width, dtype=dtype)
        lead = 16 if wide == "even" else 3
        pad = -(width + lead) % 16 if wide == "even" else 2
        return self(n, width + lead + pad, dtype=dtype)[:, lead:lead + width]


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


LENS = {
    "one": [1],
    "two": [2],
    "long": [333],
    "ragged": [0, 1, 5, 0, 2, 64, 3, 0, 129, 1, 1, 31, 0],
    "tile": [16, 64, 128, 15, 17, 0],
    "empty": [0, 0, 0],
}


# ---------------------------------------------------------------- convolution

def conv_args(lens, C, K, dtype, bias, state, wide, seed=0):
    d = Draw(seed)
    T, N = int(sum(lens)), len(lens)
    return dict(x=d.rows(T, C, dtype, wide), weight=d(C, K, std=K ** -0.5),
                bias=d(C) if bias else None, init=d(N, K - 1, C, dtype=dtype) if state else None)


def check_conv(lens, C, K, dtype, bias, state, act, wide, seed=0):
    a = conv_args(lens, C, K, dtype, bias, state, wide, seed)
    cu = cu_of(lens)
    fin = torch.full((len(lens), K - 1, C), float("nan"), dtype=dtype, device="cuda")
    out, fin2 = gdn.gdn_short_conv(a["x"], a["weight"], cu, bias=a["bias"],
                                   initial_state=a["init"], activation=act, final_state=fin)
    assert fin2 is fin
    w_out, w_err, w_fin = ref.conv(f64(a["x"]), f64(a["weight"]), cu.tolist(), f64(a["bias"]),
                                   f64(a["init"]), act, u_of(dtype))
    near(out, w_out, w_err, "out")
    near(fin, w_fin, np.zeros_like(w_fin), "final state")


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [2, 4])
def test_conv_lengths(lens, dtype, K):
    check_conv(LENS[lens], 48, K, TYPES[dtype], True, True, "silu", False)


@pytest.mark.parametrize("K", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("C", [1, 37, 8, 264, 1040])
def test_conv_widths(K, C):
    check_conv(LENS["ragged"], C, K, torch.bfloat16, False, K % 2 == 0, None, False)
    check_conv(LENS["ragged"], C, K, torch.float32, True, K % 2 == 1, "silu", False)


@pytest.mark.parametrize("C", [2, 4, 6, 12, 20, 516, 1028])
@pytest.mark.parametrize("K", [3, 4, 8])
def test_conv_narrow_words(K, C):
    """Rows of 16-bit elements at 4- and 8-byte boundaries."""
    check_conv(LENS["ragged"], C, K, torch.bfloat16, True, True, "silu", False)


@pytest.mark.parametrize("wide", ["even", "odd"])
@pytest.mark.parametrize("dtype", TYPES)
def test_conv_strided_rows(wide, dtype):
    check_conv(LENS["tile"], 80, 4, TYPES[dtype], True, True, "silu", wide)


def test_conv_many_sequences():
    check_conv([3, 0, 1, 7] * 100, 24, 4, torch.bfloat16, False, True, "silu", False)


@pytest.mark.parametrize("lens", ["one", "ragged", "long"])
def test_conv_state_in_place(lens):
    """final_state may be the initial state: the result is that of two buffers."""
    lens = LENS[lens]
    for dtype in TYPES.values():
        a = conv_args(lens, 40, 4, dtype, False, True, False)
        cu = cu_of(lens)
        out, fin = gdn.gdn_short_conv(a["x"], a["weight"], cu, initial_state=a["init"],
                                      output_final_state=True)
        both = a["init"].clone()
        out2, _ = gdn.gdn_short_conv(a["x"], a["weight"], cu, initial_state=both,
                                     final_state=both)
        assert torch.equal(out, out2) and torch.equal(fin, both)


def test_conv_in_two_calls_equals_one():
    """Cutting a sequence and carrying the state gives the same bits."""
    a = conv_args([100], 72, 4, torch.bfloat16, True, True, False)
    x = a["x"]
    out, fin = gdn.gdn_short_conv(x, a["weight"], cu_of([100]), bias=a["bias"],
                                  initial_state=a["init"], activation="silu",
                                  output_final_state=True)
    for cut in (1, 2, 50, 99):
        o1, s1 = gdn.gdn_short_conv(x[:cut], a["weight"], cu_of([cut]), bias=a["bias"],
                                    initial_state=a["init"], activation="silu",
                                    output_final_state=True)
        o2, s2 = gdn.gdn_short_conv(x[cut:], a["weight"], cu_of([100 - cut]), bias=a["bias"],
                                    initial_state=s1, activation="silu", output_final_state=True)
        assert torch.equal(torch.cat([o1, o2]), out) and torch.equal(s2, fin)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C", [1, 37, 264])
@pytest.mark.parametrize("N", [1, 5, 700])
def test_conv_step(dtype, C, N):
    """One token of each sequence, in place and apart, is a convolution of
    sequences of one token."""
    dt = TYPES[dtype]
    for K, wide in ((2, False), (4, "odd"), (8, "even")):
        a = conv_args([1] * N, C, K, dt, True, True, wide)
        w_out, w_err, w_fin = ref.conv(f64(a["x"]), f64(a["weight"]), list(range(N + 1)),
                                       f64(a["bias"]), f64(a["init"]), "silu", u_of(dt))
        new = torch.full_like(a["init"], float("nan"))
        old = a["init"].clone()
        out = gdn.gdn_short_conv_step(a["x"], a["weight"], a["init"], bias=a["bias"],
                                      activation="silu", new_state=new)
        near(out, w_out, w_err, "out")
        near(new, w_fin, np.zeros_like(w_fin), "new state")
        assert torch.equal(old, a["init"])
        out2 = gdn.gdn_short_conv_step(a["x"], a["weight"], a["init"], bias=a["bias"],
                                       activation="silu")
        assert torch.equal(out, out2) and torch.equal(a["init"], new)


# ----------------------------------------------------------------------- scan

def scan_args(rows, seqs, d, S, G, dtype, gate, skip, state, wide, seed=0):
    r = Draw(seed)
    step = np.exp(r.rng.uniform(np.log(1e-3), np.log(1e-1), d))
    f = lambda v: torch.from_numpy(v).float().cuda()  # noqa: E731
    return dict(x=r.rows(rows, d, dtype, wide), dt=r.rows(rows, d, dtype, wide) * 0.5
                if not wide else r.rows(rows, d, dtype, wide),
                A=-f(np.arange(1, S + 1) * r.rng.uniform(0.8, 1.25, (d, S))),
                B=r.rows(rows, G * S, dtype, wide).unflatten(1, (G, S)),
                C=r.rows(rows, G * S, dtype, wide).unflatten(1, (G, S)),
                D=r(d) if skip else None, z=r.rows(rows, d, dtype, wide) if gate else None,
                dt_bias=f(step + np.log(-np.expm1(-step))),
                init=r(seqs, d, S) if state else None)


def scan_ref(a, cu, dtype, softplus=True):
    return ref.scan(f64(a["x"]), f64(a["dt"]), f64(a["A"]), f64(a["B"]), f64(a["C"]), cu,
                    f64(a["D"]), f64(a["z"]), f64(a["dt_bias"]), softplus, f64(a["init"]),
                    u_of(dtype))


def run_scan(a, cu, softplus=True, **kw):
    return gdn.gdn_selective_scan(a["x"], a["dt"], a["A"], a["B"], a["C"], cu, D=a["D"],
                                  z=a["z"], dt_bias=a["dt_bias"], dt_softplus=softplus,
                                  initial_state=a["init"], **kw)


def check_scan(lens, d, S, G, dtype, gate=True, skip=True, state=True, wide=False, seed=0):
    a = scan_args(int(sum(lens)), len(lens), d, S, G, dtype, gate, skip, state, wide, seed)
    cu = cu_of(lens)
    # Scratch and results start as NaN: reads of what the call did not write show.
    need = gdn.gdn_selective_scan_workspace_size(len(lens), int(sum(lens)), d, S, G, dtype)
    ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    fin = torch.full((len(lens), d, S), float("nan"), device="cuda")
    out, _ = run_scan(a, cu, final_state=fin, workspace=ws)
    w_out, w_err, w_fin, f_err = scan_ref(a, cu.tolist(), dtype)
    near(out, w_out, w_err, "out")
    near(fin, w_fin, f_err, "final state")


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("state", [False, True])
def test_scan_lengths(lens, dtype, state):
    check_scan(LENS[lens], 48, 16, 1, TYPES[dtype], state=state)


@pytest.mark.parametrize("S", [1, 3, 4, 5, 8, 13, 16, 20, 32, 33, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_scan_states(S, dtype):
    check_scan(LENS["ragged"], 40, S, 1, TYPES[dtype])
    check_scan([70, 70], 37, S, 1, TYPES[dtype], gate=False, skip=False)


@pytest.mark.parametrize("d,G", [(1, 1), (2, 2), (30, 2), (257, 1), (264, 3), (520, 1), (520, 4)])
@pytest.mark.parametrize("dtype", TYPES)
def test_scan_channels_and_groups(d, G, dtype):
    check_scan([150, 0, 43], d, 16, G, TYPES[dtype])


@pytest.mark.parametrize("wide", ["even", "odd"])
@pytest.mark.parametrize("dtype", TYPES)
def test_scan_strided_rows(wide, dtype):
    check_scan(LENS["tile"], 72, 16, 1, TYPES[dtype], wide=wide)
    check_scan(LENS["tile"], 72, 7, 3, TYPES[dtype], wide=wide)


@pytest.mark.parametrize("d,G", [(1, 1), (3, 1), (3, 3), (5, 1), (9, 3), (67, 1), (130, 2)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("wide", [False, "even", "odd"])
def test_scan_unaligned_rows(d, G, dtype, wide):
    """Rows that start anywhere in a 16-byte word, the tensor's first included."""
    check_scan([1, 40, 2, 21], d, 4, G, TYPES[dtype], wide=wide)
    check_scan([230], d, 5, G, TYPES[dtype], gate=False, wide=wide)


@pytest.mark.parametrize("d,G,T", [(2048, 1, 1200), (2048, 1, 520), (623, 1, 700), (1246, 2, 900)])
def test_scan_windows_joined_in_runs(d, G, T):
    """Window counts that are joined in one, four and sixteen runs, and narrow blocks."""
    check_scan([T // 2, 0, T - T // 2], d, 3, G, torch.bfloat16)
    check_scan([T], d, 3, G, torch.float32, gate=False)


def test_scan_without_softplus_and_bias():
    """Steps taken as they are, negative ones among them, with growing states."""
    a = scan_args(40, 1, 24, 8, 1, torch.float32, True, True, True, False)
    a["dt"], a["dt_bias"] = 0.1 * a["dt"], None
    out, fin = run_scan(a, cu_of([40]), softplus=False, output_final_state=True)
    w_out, w_err, w_fin, f_err = scan_ref(a, [0, 40], torch.float32, softplus=False)
    near(out, w_out, w_err, "out")
    near(fin, w_fin, f_err, "final state")


def test_scan_softplus_over_its_range():
    """The step from 1e-30 to 90: its relative accuracy shows in the state."""
    n = 512
    a = scan_args(1, 1, n, 1, 1, torch.float32, False, False, False, False)
    a["dt"] = torch.linspace(-69.0, 90.0, n, device="cuda")[None]
    a["dt_bias"] = None
    a["x"], a["B"] = torch.ones_like(a["x"]), torch.ones_like(a["B"])
    _, fin = run_scan(a, cu_of([1]), output_final_state=True)
    want = np.logaddexp(0.0, f64(a["dt"]))[0][None, :, None]
    near(fin, want, want * (2.0 * np.abs(f64(a["dt"]))[0][None, :, None] + 14.0) * ref.U, "step")


@pytest.mark.parametrize("lens", ["one", "ragged", "long", "tile"])
def test_scan_state_in_place(lens):
    lens = LENS[lens]
    a = scan_args(int(sum(lens)), len(lens), 40, 16, 1, torch.bfloat16, True, True, True, False)
    cu = cu_of(lens)
    out, fin = run_scan(a, cu, output_final_state=True)
    both = a["init"].clone()
    out2, _ = run_scan(dict(a, init=both), cu, final_state=both)
    assert torch.equal(out, out2) and torch.equal(fin, both)


def test_scan_infinities_stay_in_their_sequence():
    """NaN and infinities of one sequence reach no other, and a sequence's
    later tokens only."""
    lens = [90, 1, 200, 40]
    a = scan_args(sum(lens), 4, 40, 16, 1, torch.bfloat16, True, True, True, False)
    cu = cu_of(lens)
    out, fin = run_scan(a, cu, output_final_state=True)
    x = a["x"].clone()
    x[90] = float("inf")
    x[91 + 150] = float("nan")
    out2, fin2 = run_scan(dict(a, x=x), cu, output_final_state=True)
    assert torch.equal(out[:90], out2[:90]) and torch.equal(out[291:], out2[291:])
    assert torch.equal(out[91:241], out2[91:241])
    assert torch.equal(fin[[0, 3]], fin2[[0, 3]])
    assert not torch.isfinite(out2[241:291].float()).any()
    assert torch.isnan(fin2[2]).all() and not torch.isfinite(fin2[1]).any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("S", [1, 5, 8, 16, 24, 50, 64])
@pytest.mark.parametrize("N", [1, 3, 130])
def test_scan_step(dtype, S, N):
    dt = TYPES[dtype]
    for d, G, wide in ((1, 1, False), (37, 1, "odd"), (96, 2, "even")):
        a = scan_args(N, N, d, S, G, dt, True, True, True, wide)
        w_out, w_err, w_fin, f_err = scan_ref(a, list(range(N + 1)), dt)
        kw = dict(D=a["D"], z=a["z"], dt_bias=a["dt_bias"], dt_softplus=True)
        old = a["init"].clone()
        new = torch.full_like(old, float("nan"))
        out = gdn.gdn_selective_scan_step(a["x"], a["dt"], a["A"], a["B"], a["C"], a["init"],
                                          new_state=new, **kw)
        near(out, w_out, w_err, "out")
        near(new, w_fin, f_err, "new state")
        assert torch.equal(old, a["init"])
        out2 = gdn.gdn_selective_scan_step(a["x"], a["dt"], a["A"], a["B"], a["C"], a["init"],
                                           **kw)
        assert torch.equal(out, out2) and torch.equal(a["init"], new)


def test_scan_steps_follow_a_prompt():
    """A prompt, then single tokens from its final state, is one longer prompt."""
    a = scan_args(150, 1, 72, 16, 1, torch.float32, True, True, False, False)
    w_out, w_err, w_fin, f_err = scan_ref(a, [0, 150], torch.float32)
    head = {k: v[:140] if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
    out, state = run_scan(head, cu_of([140]), output_final_state=True)
    outs = [out]
    for t in range(140, 150):
        at = slice(t, t + 1)
        outs.append(gdn.gdn_selective_scan_step(
            a["x"][at], a["dt"][at], a["A"], a["B"][at], a["C"][at], state, D=a["D"],
            z=a["z"][at], dt_bias=a["dt_bias"], dt_softplus=True))
    near(torch.cat(outs), w_out, w_err, "out")
    near(state, w_fin, f_err, "state")


# ----------------------------------------------------------------------- norm

def check_norm(rows, dim, dtype, rdt, weight, gate, first, residual, nxt, act="silu", wide=False):
    d = Draw(rows + dim)
    a = dict(y=d.rows(rows, dim, dtype, wide), weight=d(dim, mean=1.0, std=0.2) if weight else None,
             gate=d.rows(rows, dim, dtype, wide) if gate else None,
             residual=d.rows(rows, dim, rdt, wide) if residual else None,
             next_weight=d(dim, mean=1.0, std=0.2) if nxt else None)
    kw = dict(activation=act, gate_first=first, scale=0.75, eps=1e-5)
    out = torch.full((rows, dim), float("nan"), dtype=rdt, device="cuda")
    out, got_next = gdn.gdn_norm_gate_residual(**a, **kw, out=out)
    want = ref.norm(*(f64(a[k]) for k in ("y", "weight", "gate", "residual", "next_weight")),
                    act=act, gate_first=first, scale=0.75, eps=1e-5, u_out=u_of(rdt),
                    u_next=u_of(dtype))
    near(out, want[0], want[1], "out")
    assert (got_next is None) == (not nxt)
    if nxt:
        near(got_next, want[2], want[3], "next")


@pytest.mark.parametrize("dim", [1, 2, 7, 8, 31, 64, 100, 128, 250, 256, 264, 511, 1000, 1024,
                                 2049, 4096, 4104, 8200, 12289, 16384])
@pytest.mark.parametrize("types", ["bf16-bf16", "bf16-f32", "f32-f32"])
def test_norm_dims(dim, types):
    dt, rdt = (TYPES[k] for k in types.split("-"))
    check_norm(5, dim, dt, rdt, True, True, False, True, True)


@pytest.mark.parametrize("gate,first", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("nxt", [False, True])
def test_norm_parts(gate, first, weight, residual, nxt):
    for act in ("silu", "sigmoid", None):
        check_norm(3, 136, torch.bfloat16, torch.bfloat16, weight, gate, first, residual, nxt, act)
        check_norm(3, 135, torch.float32, torch.float32, weight, gate, first, residual, nxt, act)


@pytest.mark.parametrize("rows", [1, 2, 9, 1000])
@pytest.mark.parametrize("wide", [False, "even", "odd"])
def test_norm_rows_and_strides(rows, wide):
    check_norm(rows, 128, torch.bfloat16, torch.float32, True, True, True, True, True, wide=wide)
    check_norm(rows, 600, torch.bfloat16, torch.bfloat16, True, True, False, True, True, wide=wide)


@pytest.mark.parametrize("dim", [4, 12, 100, 260, 1028, 3788, 4100])
@pytest.mark.parametrize("types", ["bf16-bf16", "bf16-f32"])
@pytest.mark.parametrize("wide", [False, "even"])
def test_norm_words_of_four(dim, types, wide):
    """Rows of 16-bit elements at 8-byte boundaries only."""
    dt, rdt = (TYPES[k] for k in types.split("-"))
    check_norm(7, dim, dt, rdt, True, True, True, True, True, wide=wide)


@pytest.mark.parametrize("rows,dim", [(700, 8200), (500, 8203), (500, 9002), (2000, 4100),
                                      (1300, 4101), (200, 16384), (3000, 1028)])
@pytest.mark.parametrize("types", ["bf16-bf16", "bf16-f32", "f32-f32"])
@pytest.mark.parametrize("parts", ["all", "residual", "gate"])
def test_norm_long_rows_in_turn(rows, dim, types, parts):
    """Blocks that take several long rows, the next ones on their way."""
    dt, rdt = (TYPES[k] for k in types.split("-"))
    check_norm(rows, dim, dt, rdt, True, parts != "residual", False, parts != "gate",
               parts != "residual", wide="odd" if parts == "gate" else False)


def test_norm_long_rows_in_place():
    """out over y, next over the gate, where later rows are copied ahead."""
    d = Draw(4)
    for rows, dim in ((700, 8200), (700, 9001), (400, 9002)):
        y, g, r = (d(rows, dim, dtype=torch.bfloat16) for _ in range(3))
        w, v = d(dim), d(dim)
        out, nxt = gdn.gdn_norm_gate_residual(y, w, g, r, v)
        y2, g2 = y.clone(), g.clone()
        o, n = gdn.gdn_norm_gate_residual(y2, w, g2, r, v, out=y2, next_out=g2)
        assert torch.equal(o, out) and torch.equal(n, nxt)


def test_norm_in_place():
    """out over y or residual, next over y or gate: the bits of two buffers."""
    d = Draw(3)
    for dim in (100, 128, 4096):
        y, g, r = (d(6, dim, dtype=torch.bfloat16) for _ in range(3))
        w, v = d(dim), d(dim)
        out, nxt = gdn.gdn_norm_gate_residual(y, w, g, r, v)
        for names in (("y", "gate"), ("residual", "y"), ("residual", "gate")):
            t = dict(y=y.clone(), gate=g.clone(), residual=r.clone())
            o, n = gdn.gdn_norm_gate_residual(**t, weight=w, next_weight=v, out=t[names[0]],
                                              next_out=t[names[1]])
            assert torch.equal(o, out) and torch.equal(n, nxt)


def test_norm_zero_rows_and_zero_values():
    """No rows; rows of zeros (the norm is eps's alone) and their next norm."""
    w = torch.ones(64, device="cuda")
    y = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    out, nxt = gdn.gdn_norm_gate_residual(y, w, next_weight=w)
    assert out.shape == nxt.shape == (0, 64)
    y = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    out, nxt = gdn.gdn_norm_gate_residual(y, w, gate=y, residual=y, next_weight=w)
    assert not out.any() and not nxt.any()


def test_norm_gate_extremes():
    """Gates far out: silu and sigmoid saturate without overflow."""
    g = torch.tensor([[-3e38, -200.0, -90.0, 0.0, 90.0, 200.0, 3e38, 1.0]], device="cuda")
    y = torch.ones_like(g)
    out, _ = gdn.gdn_norm_gate_residual(y, gate=g, activation="sigmoid")
    assert out.tolist()[0][:7] == [0.0, 0.0, 0.0, 0.5, 1.0, 1.0, 1.0]
    out, _ = gdn.gdn_norm_gate_residual(y, gate=g, activation="silu")
    assert out[0, 0] == 0 and out[0, 1] == 0 and out[0, 4] == 90 and out[0, 6] == g[0, 6]


# ------------------------------------------------------------------- streams

def test_calls_run_on_the_given_stream():
    """Every operator on a side stream, after that stream's own producer."""
    side = torch.cuda.Stream()
    a = scan_args(300, 1, 64, 16, 1, torch.bfloat16, True, True, True, False)
    w = Draw(1)(64, 4)
    cu = cu_of([300])
    x = a["x"]
    want_c, _ = gdn.gdn_short_conv(x, w, cu, activation="silu")
    want_s, want_f = run_scan(dict(a, x=want_c), cu, output_final_state=True)
    want_n, _ = gdn.gdn_norm_gate_residual(want_s, torch.ones(64, device="cuda"))
    torch.cuda.synchronize()
    one = torch.ones(64, device="cuda")
    late = torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
        c, _ = gdn.gdn_short_conv(late, w, cu, activation="silu")
        s, f = run_scan(dict(a, x=c), cu, output_final_state=True)
        n, _ = gdn.gdn_norm_gate_residual(s, one)
    side.synchronize()
    assert torch.equal(c, want_c) and torch.equal(s, want_s)
    assert torch.equal(f, want_f) and torch.equal(n, want_n)
