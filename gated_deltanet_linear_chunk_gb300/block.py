"""Binding of the operators beside the layer in a hybrid block (C ABI in
``include/gdn_block.h``): the short causal convolution of the projections, the
selective state space scan, and the norms around a block fused with its gate
and residual.  As for the layer itself, this module only checks tensors and
marshals pointers and the current stream; every step runs in the library.
"""
from __future__ import annotations

import ctypes
import functools
import threading
from typing import Optional, Tuple

import torch

GDN_ACT_NONE = 0
GDN_ACT_SILU = 1
GDN_ACT_SIGMOID = 2
_ACTIVATIONS = {None: GDN_ACT_NONE, "none": GDN_ACT_NONE, "silu": GDN_ACT_SILU,
                "sigmoid": GDN_ACT_SIGMOID}
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}  # gdn_dtype

_P, _I32, _I64, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class ConvProblem(ctypes.Structure):
    """Mirror of ``gdn_conv_problem`` in include/gdn_block.h."""

    _fields_ = [("num_seqs", _I32), ("total_tokens", _I64), ("channels", _I32), ("width", _I32),
                ("dtype", _I32), ("activation", _I32), ("x_stride", _I64), ("out_stride", _I64)]


class SsmProblem(ctypes.Structure):
    """Mirror of ``gdn_ssm_problem`` in include/gdn_block.h."""

    _fields_ = [("num_seqs", _I32), ("total_tokens", _I64), ("channels", _I32),
                ("state_dim", _I32), ("num_groups", _I32), ("dtype", _I32),
                ("dt_softplus", _I32), ("x_stride", _I64), ("dt_stride", _I64),
                ("b_stride", _I64), ("c_stride", _I64), ("z_stride", _I64), ("out_stride", _I64),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class NormProblem(ctypes.Structure):
    """Mirror of ``gdn_norm_problem`` in include/gdn_block.h."""

    _fields_ = [("rows", _I64), ("dim", _I32), ("dtype", _I32), ("residual_dtype", _I32),
                ("activation", _I32), ("gate_first", _I32), ("eps", _F32), ("scale", _F32),
                ("y_stride", _I64), ("gate_stride", _I64), ("residual_stride", _I64),
                ("out_stride", _I64), ("next_stride", _I64)]


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of this module's entry points."""
    conv, ssm = ctypes.POINTER(ConvProblem), ctypes.POINTER(SsmProblem)
    for name, problem, pointers in (("gdn_short_conv", conv, 8), ("gdn_short_conv_step", conv, 7),
                                    ("gdn_selective_scan", ssm, 13),
                                    ("gdn_selective_scan_step", ssm, 12),
                                    ("gdn_norm_gate_residual",
                                     ctypes.POINTER(NormProblem), 8)):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = [problem] + [_P] * pointers
    lib.gdn_selective_scan_workspace_size.restype = ctypes.c_size_t
    lib.gdn_selective_scan_workspace_size.argtypes = [ssm]


from . import (  # noqa: E402  (the package's helpers, defined before this import)
    GDNError, _check, _stream_obj, _workspace, _workspaces, library)


def _rows(t: torch.Tensor, name: str, dtype, shape, dev: int) -> int:
    """Checks a token-major tensor on device `dev`, whose rows may be strided,
    and returns its row stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if dev < 0 or t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}: all tensors of a call must be on one CUDA "
                         "device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    stride = t.stride()
    width, whole = shape[1], stride[1] == 1 or shape[1] == 1
    if len(shape) == 3:  # [rows, groups, states]
        width *= shape[2]
        whole = (shape[1] == 1 or stride[1] == shape[2]) and (shape[2] == 1 or stride[2] == 1)
    if whole and (shape[0] <= 1 or stride[0] >= width):
        return stride[0]
    if t.numel() == 0:  # no elements: the strides mean nothing
        return width
    raise ValueError(f"{name} must be contiguous within its rows, and its rows must not overlap "
                     f"(shape {tuple(shape)}, strides {stride})")


def _ptr(t: Optional[torch.Tensor], name: str, dtype, shape, dev: int) -> Optional[int]:
    """Checks an optional contiguous tensor on device `dev`; its pointer."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or \
            not t.is_contiguous():
        _check(t, name, dtype, shape)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}: all tensors of a call must be on one CUDA "
                         "device")
    return t.data_ptr()


def _activation(name) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError(f"unknown activation {name!r}")
    return _ACTIVATIONS[name]


def _dtype(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype} of {name}")
    return _DTYPES[t.dtype]


# The handle of a device's current stream, without the stream object that
# torch.cuda.current_stream makes on every call (1 us of a step's 12).
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _call(name: str, dev: int, *args) -> None:
    """Calls an entry point on device `dev` and that device's current stream."""
    f = getattr(library(), name)
    if dev == torch.cuda.current_device():
        rc = f(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = f(*args, _raw_stream(dev))
    if rc != 0:
        raise GDNError(rc, name)


def _with_stream(f):
    """A call given a stream runs with that stream current, so that the
    results it allocates belong to that stream too."""
    @functools.wraps(f)
    def g(*args, stream=None, **kwargs):
        if stream is None:
            return f(*args, **kwargs)
        first = args[0] if args else next(iter(kwargs.values()))
        with torch.cuda.stream(_stream_obj(stream, first.device)):
            return f(*args, **kwargs)
    return g


@_with_stream
def gdn_short_conv(x: torch.Tensor, weight: torch.Tensor, cu_seqlens: torch.Tensor,
                   bias: Optional[torch.Tensor] = None,
                   initial_state: Optional[torch.Tensor] = None, activation=None,
                   out: Optional[torch.Tensor] = None,
                   final_state: Optional[torch.Tensor] = None, output_final_state: bool = False,
                   *, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Short causal depthwise convolution over packed sequences (see
    ``gdn_short_conv`` in include/gdn_block.h).  x: [T, C] bf16 or fp32, rows
    may be strided; weight: [C, K] fp32; bias: [C] fp32; cu_seqlens: [N+1]
    int32; initial_state, final_state: [N, K-1, C] in x's dtype, oldest input
    first (they may be one tensor); activation: None or "silu".  Returns (out
    [T, C], final_state), the final state when ``final_state`` is given or
    ``output_final_state`` is set."""
    code, dev = _dtype(x, "x"), x.get_device()
    T, C = shape = x.shape
    K, N = weight.shape[1], cu_seqlens.shape[0] - 1
    dt, f32, state = x.dtype, torch.float32, (N, K - 1, C)
    xs, os_ = _rows(x, "x", dt, shape, dev), C
    if out is None:
        out = torch.empty(shape, dtype=dt, device=x.device)
    else:
        os_ = _rows(out, "out", dt, shape, dev)
    if final_state is None and output_final_state:
        final_state = torch.empty(state, dtype=dt, device=x.device)
    p = ConvProblem(N, T, C, K, code, _activation(activation), xs, os_)
    _call("gdn_short_conv", dev, p, x.data_ptr(), _ptr(weight, "weight", f32, (C, K), dev),
          _ptr(bias, "bias", f32, (C,), dev),
          _ptr(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev),
          _ptr(initial_state, "initial_state", dt, state, dev), out.data_ptr(),
          _ptr(final_state, "final_state", dt, state, dev))
    return out, final_state


@_with_stream
def gdn_short_conv_step(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor,
                        bias: Optional[torch.Tensor] = None, activation=None,
                        out: Optional[torch.Tensor] = None,
                        new_state: Optional[torch.Tensor] = None, *,
                        stream=None) -> torch.Tensor:
    """``gdn_short_conv`` for one token of each sequence: x [N, C]; state
    [N, K-1, C] is updated in place, or left as it is when ``new_state`` is
    given to hold the new one.  Returns out [N, C]."""
    code, dev = _dtype(x, "x"), x.get_device()
    N, C = shape = x.shape
    K = weight.shape[1]
    dt, f32, rows = x.dtype, torch.float32, (N, K - 1, C)
    xs, os_ = _rows(x, "x", dt, shape, dev), C
    if out is None:
        out = torch.empty(shape, dtype=dt, device=x.device)
    else:
        os_ = _rows(out, "out", dt, shape, dev)
    p = ConvProblem(N, N, C, K, code, _activation(activation), xs, os_)
    old = _ptr(state, "state", dt, rows, dev)
    _call("gdn_short_conv_step", dev, p, x.data_ptr(), _ptr(weight, "weight", f32, (C, K), dev),
          _ptr(bias, "bias", f32, (C,), dev), old, out.data_ptr(),
          old if new_state is None else _ptr(new_state, "new_state", dt, rows, dev))
    return out


def _ssm(N, x, dt, A, B, C, D, z, dt_bias, dt_softplus, out):
    """Checks of what the scan and its step share: (problem, out, pointers of
    x .. dt_bias in the entry points' order)."""
    code, dev = _dtype(x, "x"), x.get_device()
    T, ch = shape = x.shape
    _, G, S = states = torch.Size((T, *B.shape[1:]))
    ty, f32 = x.dtype, torch.float32
    xs, os_ = _rows(x, "x", ty, shape, dev), ch
    if out is None:
        out = torch.empty(shape, dtype=ty, device=x.device)
    else:
        os_ = _rows(out, "out", ty, shape, dev)
    p = SsmProblem(N, T, ch, S, G, code, 1 if dt_softplus else 0, xs,
                   _rows(dt, "dt", ty, shape, dev), _rows(B, "B", ty, states, dev),
                   _rows(C, "C", ty, states, dev),
                   0 if z is None else _rows(z, "z", ty, shape, dev), os_, None, 0)
    return p, out, (x.data_ptr(), dt.data_ptr(), _ptr(A, "A", f32, (ch, S), dev), B.data_ptr(),
                    C.data_ptr(), _ptr(D, "D", f32, (ch,), dev),
                    None if z is None else z.data_ptr(),
                    _ptr(dt_bias, "dt_bias", f32, (ch,), dev))


@_with_stream
def gdn_selective_scan(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                       C: torch.Tensor, cu_seqlens: torch.Tensor,
                       D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                       dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False,
                       initial_state: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None,
                       final_state: Optional[torch.Tensor] = None,
                       output_final_state: bool = False,
                       workspace: Optional[torch.Tensor] = None, *,
                       stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Selective state space scan over packed sequences (see
    ``gdn_selective_scan`` in include/gdn_block.h).  x, dt, z: [T, channels];
    B, C: [T, groups, states] (all one dtype, bf16 or fp32; rows may be
    strided); A: [channels, states], D, dt_bias: [channels] fp32; cu_seqlens:
    [N+1] int32; states [N, channels, states] fp32 (initial and final may be
    one tensor).  Returns (out [T, channels], final_state), the final state
    when ``final_state`` is given or ``output_final_state`` is set."""
    N, f32, dev = cu_seqlens.shape[0] - 1, torch.float32, x.get_device()
    p, out, inputs = _ssm(N, x, dt, A, B, C, D, z, dt_bias, dt_softplus, out)
    state = (N, p.channels, p.state_dim)
    if final_state is None and output_final_state:
        final_state = torch.empty(state, dtype=f32, device=x.device)
    if workspace is None:
        need = library().gdn_selective_scan_workspace_size(p)
        if need:
            key = (dev, _raw_stream(dev), threading.get_ident())
            workspace = _workspaces.get(key)
            if workspace is None or workspace.numel() < need:
                workspace = _workspace(x.device, need)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the call's device")
    if workspace is not None:
        p.workspace = workspace.data_ptr()
        p.workspace_bytes = workspace.numel() * workspace.element_size()
    _call("gdn_selective_scan", dev, p, *inputs,
          _ptr(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev),
          _ptr(initial_state, "initial_state", f32, state, dev), out.data_ptr(),
          _ptr(final_state, "final_state", f32, state, dev))
    return out, final_state


def gdn_selective_scan_workspace_size(N: int, T: int, channels: int, states: int, groups: int = 1,
                                      dtype=torch.bfloat16) -> int:
    """Workspace bytes of ``gdn_selective_scan`` (0: none needed, or sizes
    that it does not support)."""
    p = SsmProblem(N, T, channels, states, groups, _DTYPES[dtype], 0, 0, 0, 0, 0, 0, 0, None, 0)
    return int(library().gdn_selective_scan_workspace_size(p))


@_with_stream
def gdn_selective_scan_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                            C: torch.Tensor, state: torch.Tensor,
                            D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                            dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False,
                            out: Optional[torch.Tensor] = None,
                            new_state: Optional[torch.Tensor] = None, *,
                            stream=None) -> torch.Tensor:
    """``gdn_selective_scan`` for one token of each sequence: x, dt, z
    [N, channels]; B, C [N, groups, states]; state [N, channels, states] fp32
    is updated in place, or left as it is when ``new_state`` is given to hold
    the new one.  Returns out [N, channels]."""
    N, f32, dev = x.shape[0], torch.float32, x.get_device()
    p, out, inputs = _ssm(N, x, dt, A, B, C, D, z, dt_bias, dt_softplus, out)
    shape = (N, p.channels, p.state_dim)
    old = _ptr(state, "state", f32, shape, dev)
    _call("gdn_selective_scan_step", dev, p, *inputs, old, out.data_ptr(),
          old if new_state is None else _ptr(new_state, "new_state", f32, shape, dev))
    return out


@_with_stream
def gdn_norm_gate_residual(y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                           gate: Optional[torch.Tensor] = None,
                           residual: Optional[torch.Tensor] = None,
                           next_weight: Optional[torch.Tensor] = None, activation="silu",
                           gate_first: bool = False, scale: float = 1.0, eps: float = 1e-6,
                           out: Optional[torch.Tensor] = None,
                           next_out: Optional[torch.Tensor] = None, *,
                           stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The norm after a block with its gate and scaled residual, and the norm
    before the next block (see ``gdn_norm_gate_residual`` in
    include/gdn_block.h):

        out  = residual + scale * weight * rms(y) * act(gate)
        next = next_weight * rms(out)

    y, gate: [R, D] bf16 or fp32, rows may be strided; residual: [R, D] in y's
    dtype or fp32, which is then also out's; weight, next_weight: [D] fp32.
    ``gate_first`` puts the gate before the norm; without ``weight`` y is not
    normed, without ``next_weight`` next is None.  ``out`` may be y or
    residual, ``next_out`` y or gate.  Returns (out, next)."""
    code, dev = _dtype(y, "y"), y.get_device()
    R, D = shape = y.shape
    dt, f32 = y.dtype, torch.float32
    stream_like = residual if residual is not None else out
    rdt = dt if stream_like is None else stream_like.dtype
    if rdt not in _DTYPES:
        raise TypeError(f"unsupported residual dtype {rdt}")
    ys, os_, ns = _rows(y, "y", dt, shape, dev), D, D
    if out is None:
        out = torch.empty(shape, dtype=rdt, device=y.device)
    else:
        os_ = _rows(out, "out", rdt, shape, dev)
    if next_weight is not None:
        if next_out is None:
            next_out = torch.empty(shape, dtype=dt, device=y.device)
        else:
            ns = _rows(next_out, "next_out", dt, shape, dev)
    elif next_out is not None:
        raise ValueError("next_out without next_weight")
    p = NormProblem(R, D, code, _DTYPES[rdt], _activation(activation), 1 if gate_first else 0,
                    eps, scale, ys, 0 if gate is None else _rows(gate, "gate", dt, shape, dev),
                    0 if residual is None else _rows(residual, "residual", rdt, shape, dev),
                    os_, ns)
    _call("gdn_norm_gate_residual", dev, p, y.data_ptr(), _ptr(weight, "weight", f32, (D,), dev),
          None if gate is None else gate.data_ptr(),
          None if residual is None else residual.data_ptr(),
          _ptr(next_weight, "next_weight", f32, (D,), dev), out.data_ptr(),
          None if next_out is None else next_out.data_ptr())
    return out, next_out
