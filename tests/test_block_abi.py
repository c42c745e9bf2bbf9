"""The block operators' C ABI and binding without a GPU: bad arguments are
refused before anything is launched."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_chunk_gb300 as gdn
from gated_deltanet_linear_chunk_gb300.block import ConvProblem, NormProblem, SsmProblem

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)
A = 0x100000  # an aligned fake device address; never dereferenced here
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return gdn.library()


def conv(lib, N=2, T=10, C=16, K=4, dtype=0, act=1, xs=16, os=16, x=A, w=A + 4096, b=None,
         cu=A + 8192, init=None, out=A + 12288, fin=None, none=False):
    p = None if none else ctypes.byref(ConvProblem(N, T, C, K, dtype, act, xs, os))
    return lib.gdn_short_conv(p, x, w, b, cu, init, out, fin, None)


def test_conv_refusals(lib):
    assert conv(lib, none=True) == INVALID
    for kw in (dict(N=-1), dict(T=-1), dict(C=0), dict(K=0), dict(T=BIG), dict(C=1 << 21),
               dict(xs=15), dict(os=15), dict(x=None), dict(out=None), dict(w=None),
               dict(cu=None), dict(out=A), dict(N=0)):
        assert conv(lib, **kw) == INVALID, kw
    for kw in (dict(K=1), dict(K=9), dict(dtype=2), dict(act=2), dict(act=-1)):
        assert conv(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(x=A + 1), dict(out=A + 1), dict(init=A + 1), dict(fin=A + 1), dict(w=A + 2),
               dict(b=A + 2), dict(cu=A + 2), dict(dtype=1, x=A + 2)):
        assert conv(lib, **kw) == MISALIGNED, kw
    assert conv(lib, N=0, T=0) == OK


def conv_step(lib, N=2, T=2, C=16, K=4, x=A, w=A + 4096, s=A + 8192, out=A + 12288,
              new=A + 16384, dtype=0):
    return lib.gdn_short_conv_step(ConvProblem(N, T, C, K, dtype, 1, 16, 16), x, w, None, s, out,
                                   new, None)


def test_conv_step_refusals(lib):
    for kw in (dict(T=3), dict(x=None), dict(w=None), dict(s=None), dict(out=None),
               dict(new=None), dict(out=A), dict(out=A + 8192), dict(out=A + 16384)):
        assert conv_step(lib, **kw) == INVALID, kw
    assert conv_step(lib, K=9) == UNSUPPORTED
    assert conv_step(lib, s=A + 1) == MISALIGNED
    assert conv_step(lib, N=0, T=0) == OK


NAMES = ("x", "dt", "a", "b", "c", "skip", "z", "bias")


def pointers(kw):
    at = dict(zip(NAMES, (A + 65536 * i for i in range(8))), **kw)
    return [at[k] for k in NAMES]


def scan(lib, N=2, T=10, D=16, S=8, G=1, dtype=0, strides=(16, 16, 8, 8, 16, 16), ws=None, wsb=0,
         cu=A + (1 << 20), init=None, out=A + (2 << 20), fin=None, none=False, **kw):
    p = None if none else ctypes.byref(SsmProblem(N, T, D, S, G, dtype, 1, *strides, ws, wsb))
    return lib.gdn_selective_scan(p, *pointers(kw), cu, init, out, fin, None)


def test_scan_refusals(lib):
    assert scan(lib, none=True) == INVALID
    for kw in (dict(N=-1), dict(T=-1), dict(T=BIG), dict(D=0), dict(S=0), dict(G=0),
               dict(x=None), dict(dt=None), dict(a=None), dict(b=None), dict(c=None),
               dict(cu=None), dict(out=None), dict(N=0), dict(out=A), dict(out=A + 65536 * 6)):
        assert scan(lib, **kw) == INVALID, kw
    for i in range(6):
        strides = [16, 16, 8, 8, 16, 16]
        strides[i] -= 1
        assert scan(lib, strides=strides) == INVALID, i
    for kw in (dict(S=65), dict(D=15, G=2), dict(dtype=2), dict(dtype=-1)):
        assert scan(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(x=A + 1), dict(b=A + 1), dict(z=A + 1), dict(a=A + 2), dict(skip=A + 2),
               dict(bias=A + 2), dict(init=A + 2), dict(fin=A + 2), dict(cu=A + 2)):
        assert scan(lib, **kw) == MISALIGNED, kw
    assert scan(lib, N=0, T=0) == OK


def test_scan_workspace(lib):
    size = lib.gdn_selective_scan_workspace_size

    def problem(T=4000, D=512, S=16, G=1, dtype=0):
        return SsmProblem(1, T, D, S, G, dtype, 1, 0, 0, 0, 0, 0, 0, None, 0)
    assert size(None) == 0
    assert size(problem(S=65)) == 0 and size(problem(D=5, G=2)) == 0 and size(problem(T=-1)) == 0
    assert size(problem(T=1)) == 0  # one token: one window
    need = size(problem())
    assert need > 0 and need % (512 * 17 * 4) == 0
    assert need == gdn.gdn_selective_scan_workspace_size(1, 4000, 512, 16)
    wide = (512, 512, 16, 16, 512, 512)
    for ws, wsb in ((None, 0), (A, need - 1), (A + 8, need)):
        assert scan(lib, N=1, T=4000, D=512, S=16, strides=wide, ws=ws, wsb=wsb) == WORKSPACE


def test_scan_step_refusals(lib):
    def step(N=2, T=2, S=8, state=A + (1 << 20), out=A + (2 << 20), new=A + (3 << 20), **kw):
        p = SsmProblem(N, T, 16, S, 1, 0, 1, 16, 16, S, S, 16, 16, None, 0)
        return lib.gdn_selective_scan_step(p, *pointers(kw), state, out, new, None)
    for kw in (dict(T=3), dict(state=None), dict(new=None), dict(out=None), dict(x=None),
               dict(out=A + (1 << 20)), dict(out=A + 65536)):
        assert step(**kw) == INVALID, kw
    assert step(S=65) == UNSUPPORTED
    assert step(state=A + 2) == MISALIGNED
    assert step(N=0, T=0) == OK


def norm(lib, R=4, D=16, dtype=0, rdt=0, act=1, eps=1e-6, strides=(16,) * 5, y=A, w=A + 4096,
         g=None, r=None, nw=None, out=A + 8192, nxt=None, none=False):
    p = None if none else ctypes.byref(NormProblem(R, D, dtype, rdt, act, 0, eps, 1.0, *strides))
    return lib.gdn_norm_gate_residual(p, y, w, g, r, nw, out, nxt, None)


def test_norm_refusals(lib):
    assert norm(lib, none=True) == INVALID
    both = dict(nw=A + 65536, nxt=A + 131072)
    for kw in (dict(R=-1), dict(D=0), dict(eps=-1.0), dict(eps=float("nan")), dict(y=None),
               dict(out=None), dict(nw=A), dict(nxt=A + 65536), dict(strides=(15,) + (16,) * 4),
               dict(strides=(16,) * 3 + (15, 16)), dict(g=A, strides=(16, 15, 16, 16, 16)),
               dict(r=A, strides=(16, 16, 15, 16, 16)),
               dict(strides=(16,) * 4 + (15,), **both),
               dict(out=A, rdt=1),                                 # over y of another type
               dict(out=A, strides=(16, 16, 16, 32, 16)),          # over y, other rows
               dict(r=A + 8192, strides=(16, 16, 32, 16, 16)),     # over residual, other rows
               dict(g=A + 8192),                                   # over the gate
               dict(nw=A + 65536, nxt=A + 8192),                   # out and next in one
               dict(r=A + 131072, **both)):                        # next over residual
        assert norm(lib, **kw) == INVALID, kw
    for kw in (dict(D=16385, strides=(16385,) * 5), dict(dtype=2), dict(rdt=2),
               dict(dtype=1, rdt=0), dict(act=3), dict(act=-1)):
        assert norm(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(y=A + 1), dict(out=A + 1), dict(w=A + 2), dict(rdt=1, r=A + 2)):
        assert norm(lib, **kw) == MISALIGNED, kw
    assert norm(lib, R=0, y=None, out=None) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_short_conv_step(x, torch.zeros(8, 4), torch.zeros(4, 3, 8))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_norm_gate_residual(x)
    with pytest.raises(TypeError):
        gdn.gdn_norm_gate_residual(x.half())
    with pytest.raises(TypeError):
        gdn.gdn_short_conv(x.int(), torch.zeros(8, 4), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_selective_scan(x, x, torch.zeros(8, 2), torch.zeros(4, 1, 2),
                               torch.zeros(4, 1, 2), torch.zeros(2, dtype=torch.int32))


def test_binding_checks_rows(lib):
    """Strided rows pass, overlapping or scattered ones do not (types, shapes
    and strides are checked before the device, so no GPU is needed to see it:
    what passes is then refused for being on the host)."""
    f32 = torch.float32

    def conv(x):
        gdn.gdn_short_conv_step(x, torch.zeros(8, 4), torch.zeros(4, 3, 8))

    def scan(B):
        x = torch.zeros(4, 8)
        gdn.gdn_selective_scan_step(x, x, torch.zeros(8, 8), B, B, torch.zeros(4, 8, 8))
    for good in (torch.zeros(4, 8), torch.zeros(4, 24)[:, 3:11]):
        with pytest.raises(ValueError, match="one CUDA device"):
            conv(good)
    for bad in (torch.zeros(8, 4).t(), torch.zeros(1, 8).expand(4, 8), torch.zeros(4, 16)[:, ::2]):
        with pytest.raises(ValueError, match="contiguous within"):
            conv(bad)
    # Rows of B are not reached before x: it is refused for its device.
    with pytest.raises(ValueError, match="one CUDA device"):
        scan(torch.zeros(4, 24)[:, 4:20].unflatten(1, (2, 8)))
    with pytest.raises(TypeError):
        conv(torch.zeros(4, 8, dtype=torch.float64))
    with pytest.raises(ValueError, match="dimensions"):
        conv(torch.zeros(4, 2, 8))
    with pytest.raises(ValueError, match="taps|tap"):
        gdn.gdn_short_conv_step(torch.zeros(4, 8, dtype=f32), torch.zeros(8, 0),
                                torch.zeros(4, 0, 8))
    with pytest.raises(TypeError, match="must be a tensor"):
        gdn.gdn_short_conv_step([1.0], torch.zeros(8, 4), torch.zeros(4, 3, 8))
    with pytest.raises(ValueError, match="activation"):
        gdn.gdn_short_conv_step(torch.zeros(4, 8), torch.zeros(8, 4), torch.zeros(4, 3, 8),
                                activation="tanh")
