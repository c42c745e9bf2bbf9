"""Binding of the operators beside the layer in a hybrid block (C ABI in
``include/gdn_block.h``): the short causal convolution of the projections, the
selective state space scan, and the norms around a block fused with its gate
and residual.  Every step runs in the library.  Tensors are checked and
marshalled by a small extension module (csrc/block_binding.cpp) rather than
here: a single token's operator takes a few microseconds, less than ten
tensors' checks do in Python (a step's call took 12 us there, 4 us through the
module; the scan's 27 and 9).
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
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


from . import build as _build  # noqa: E402
from . import GDNError, _stream_obj, library  # noqa: E402  (defined before this import)

_ENTRIES = ("gdn_short_conv", "gdn_short_conv_step", "gdn_selective_scan",
            "gdn_selective_scan_step", "gdn_selective_scan_workspace_size",
            "gdn_norm_gate_residual")
_native = None


def _binding():
    """The extension module that checks tensors and calls the entry points;
    raises if it, or the library, has not been built."""
    global _native
    if _native is None:
        lib, path = library(), _build.binding_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"the binding {path} is missing: build it first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        spec = importlib.util.spec_from_file_location("gdn_block_binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(GDNError, *[ctypes.cast(getattr(lib, e), _P).value for e in _ENTRIES])
        _native = module
    return _native


def _activation(name) -> int:
    code = _ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"unknown activation {name!r}")
    return code


def gdn_short_conv(x: torch.Tensor, weight: torch.Tensor, cu_seqlens: torch.Tensor,
                   bias: Optional[torch.Tensor] = None,
                   initial_state: Optional[torch.Tensor] = None, activation=None,
                   out: Optional[torch.Tensor] = None,
                   final_state: Optional[torch.Tensor] = None, output_final_state: bool = False,
                   stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Short causal depthwise convolution over packed sequences (see
    ``gdn_short_conv`` in include/gdn_block.h).  x: [T, C] bf16 or fp32, rows
    may be strided; weight: [C, K] fp32; bias: [C] fp32; cu_seqlens: [N+1]
    int32; initial_state, final_state: [N, K-1, C] in x's dtype, oldest input
    first (they may be one tensor); activation: None or "silu".  Returns (out
    [T, C], final_state), the final state when ``final_state`` is given or
    ``output_final_state`` is set.  With ``stream`` the call runs on it, and
    its results belong to it."""
    if stream is not None:
        with torch.cuda.stream(_stream_obj(stream, x.device)):
            return gdn_short_conv(x, weight, cu_seqlens, bias, initial_state, activation, out,
                                  final_state, output_final_state)
    return (_native or _binding()).short_conv(x, weight, cu_seqlens, bias, initial_state,
                                              _activation(activation), out, final_state,
                                              output_final_state)


def gdn_short_conv_step(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor,
                        bias: Optional[torch.Tensor] = None, activation=None,
                        out: Optional[torch.Tensor] = None,
                        new_state: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``gdn_short_conv`` for one token of each sequence: x [N, C]; state
    [N, K-1, C] is updated in place, or left as it is when ``new_state`` is
    given to hold the new one.  Returns out [N, C]."""
    if stream is not None:
        with torch.cuda.stream(_stream_obj(stream, x.device)):
            return gdn_short_conv_step(x, weight, state, bias, activation, out, new_state)
    return (_native or _binding()).short_conv_step(x, weight, state, bias,
                                                   _activation(activation), out, new_state)


def gdn_selective_scan(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                       C: torch.Tensor, cu_seqlens: torch.Tensor,
                       D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                       dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False,
                       initial_state: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None,
                       final_state: Optional[torch.Tensor] = None,
                       output_final_state: bool = False,
                       workspace: Optional[torch.Tensor] = None,
                       stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Selective state space scan over packed sequences (see
    ``gdn_selective_scan`` in include/gdn_block.h).  x, dt, z: [T, channels];
    B, C: [T, groups, states] (all one dtype, bf16 or fp32; rows may be
    strided); A: [channels, states], D, dt_bias: [channels] fp32; cu_seqlens:
    [N+1] int32; states [N, channels, states] fp32 (initial and final may be
    one tensor).  ``workspace`` is scratch of at least
    ``gdn_selective_scan_workspace_size`` bytes, by default taken from the
    caching allocator for the call.  Returns (out [T, channels], final_state),
    the final state when ``final_state`` is given or ``output_final_state`` is
    set."""
    if stream is not None:
        with torch.cuda.stream(_stream_obj(stream, x.device)):
            return gdn_selective_scan(x, dt, A, B, C, cu_seqlens, D, z, dt_bias, dt_softplus,
                                      initial_state, out, final_state, output_final_state,
                                      workspace)
    return (_native or _binding()).selective_scan(
        x, dt, A, B, C, cu_seqlens, D, z, dt_bias, dt_softplus, initial_state, out, final_state,
        output_final_state, workspace)


def gdn_selective_scan_workspace_size(N: int, T: int, channels: int, states: int, groups: int = 1,
                                      dtype=torch.bfloat16) -> int:
    """Workspace bytes of ``gdn_selective_scan`` (0: none needed, or sizes
    that it does not support)."""
    p = SsmProblem(N, T, channels, states, groups, _DTYPES[dtype], 0, 0, 0, 0, 0, 0, 0, None, 0)
    return int(library().gdn_selective_scan_workspace_size(p))


def gdn_selective_scan_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                            C: torch.Tensor, state: torch.Tensor,
                            D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                            dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False,
                            out: Optional[torch.Tensor] = None,
                            new_state: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """``gdn_selective_scan`` for one token of each sequence: x, dt, z
    [N, channels]; B, C [N, groups, states]; state [N, channels, states] fp32
    is updated in place, or left as it is when ``new_state`` is given to hold
    the new one.  Returns out [N, channels]."""
    if stream is not None:
        with torch.cuda.stream(_stream_obj(stream, x.device)):
            return gdn_selective_scan_step(x, dt, A, B, C, state, D, z, dt_bias, dt_softplus,
                                           out, new_state)
    return (_native or _binding()).selective_scan_step(x, dt, A, B, C, state, D, z, dt_bias,
                                                       dt_softplus, out, new_state)


def gdn_norm_gate_residual(y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                           gate: Optional[torch.Tensor] = None,
                           residual: Optional[torch.Tensor] = None,
                           next_weight: Optional[torch.Tensor] = None, activation="silu",
                           gate_first: bool = False, scale: float = 1.0, eps: float = 1e-6,
                           out: Optional[torch.Tensor] = None,
                           next_out: Optional[torch.Tensor] = None,
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
    if stream is not None:
        with torch.cuda.stream(_stream_obj(stream, y.device)):
            return gdn_norm_gate_residual(y, weight, gate, residual, next_weight, activation,
                                          gate_first, scale, eps, out, next_out)
    return (_native or _binding()).norm_gate_residual(
        y, weight, gate, residual, next_weight, _activation(activation), gate_first, scale, eps,
        out, next_out)
