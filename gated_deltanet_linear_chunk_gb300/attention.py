"""Binding of the attention layers' operators (C ABI in
``include/gdn_attention.h``): norms of queries and keys for each head with
their rotation by position, a paged cache that new keys and values are appended
to on the way, and the attention of each sequence's newest tokens over it.
Every step runs in the library; tensors are checked and marshalled by the
extension module of the block operators.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple, Union

import torch

_P, _I32, _I64, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class RopeProblem(ctypes.Structure):
    """Mirror of ``gdn_rope_problem`` in include/gdn_attention.h."""

    _fields_ = [("total_tokens", _I64), ("q_heads", _I32), ("kv_heads", _I32), ("head_dim", _I32),
                ("dtype", _I32), ("rotary_dim", _I32), ("interleaved", _I32), ("num_axes", _I32),
                ("freq_axis", ctypes.POINTER(ctypes.c_uint8)), ("eps", _F32),
                ("axis_stride", _I64), ("q_stride", _I64), ("q_head_stride", _I64),
                ("k_stride", _I64), ("k_head_stride", _I64), ("v_stride", _I64),
                ("v_head_stride", _I64), ("q_out_stride", _I64), ("q_out_head_stride", _I64),
                ("k_out_stride", _I64), ("k_out_head_stride", _I64)]


class PagedCache(ctypes.Structure):
    """Mirror of ``gdn_paged_cache`` in include/gdn_attention.h."""

    _fields_ = [("k", _P), ("v", _P), ("dtype", _I32), ("num_pages", _I64), ("page_size", _I32),
                ("k_page_stride", _I64), ("k_token_stride", _I64), ("k_head_stride", _I64),
                ("v_page_stride", _I64), ("v_token_stride", _I64), ("v_head_stride", _I64),
                ("k_scale", _P), ("v_scale", _P), ("num_seqs", _I32), ("max_pages", _I32),
                ("page_table", _P), ("table_stride", _I64), ("seq_lens", _P)]


class AttentionProblem(ctypes.Structure):
    """Mirror of ``gdn_attention_problem`` in include/gdn_attention.h."""

    _fields_ = [("new_tokens", _I32), ("q_heads", _I32), ("kv_heads", _I32), ("head_dim", _I32),
                ("dtype", _I32), ("scale", _F32), ("q_stride", _I64), ("q_head_stride", _I64),
                ("gate_stride", _I64), ("gate_head_stride", _I64), ("out_stride", _I64),
                ("out_head_stride", _I64), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of this module's entry points."""
    rope, cache = ctypes.POINTER(RopeProblem), ctypes.POINTER(PagedCache)
    attention = ctypes.POINTER(AttentionProblem)
    for name, types in (("gdn_qk_norm_rope", [rope] + [_P] * 9),
                        ("gdn_paged_append", [rope, cache] + [_P] * 10),
                        ("gdn_paged_attention", [attention, cache] + [_P] * 5)):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = types
    lib.gdn_paged_attention_workspace_size.restype = ctypes.c_size_t
    lib.gdn_paged_attention_workspace_size.argtypes = [attention, cache]


from . import GDN_BF16, GDN_E4M3, GDN_F32, _stream_obj, block, library  # noqa: E402

_ENTRIES = ("gdn_qk_norm_rope", "gdn_paged_append", "gdn_paged_attention",
            "gdn_paged_attention_workspace_size")
_CACHE_DTYPES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32, torch.float8_e4m3fn: GDN_E4M3}
_native = None


def _binding():
    """The extension module, with this module's entry points bound."""
    global _native
    if _native is None:
        module, lib = block._binding(), library()
        module.bind_attention(*[ctypes.cast(getattr(lib, e), _P).value for e in _ENTRIES])
        _native = module
    return _native


def gdn_qk_norm_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor] = None,
                     positions: Optional[torch.Tensor] = None,
                     inv_freq: Optional[torch.Tensor] = None,
                     q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     axes: Optional[Sequence[int]] = None, interleaved: bool = False,
                     q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """RMS norms of queries and keys for each head with their rotation by
    position, in one pass (see ``gdn_qk_norm_rope`` in
    include/gdn_attention.h).  q: [T, Hq, D], k: [T, Hk, D] bf16 or fp32 (either
    may be None), strided between tokens and heads; positions: [T] int32, or
    [axes, T] with ``axes`` naming the axis of each pair; inv_freq: [pairs]
    fp32, radians per position (None: no rotation); q_weight, k_weight: [D]
    fp32 (None: no norm).  The first 2 * pairs elements of a head are rotated:
    element i with i + pairs, or ``interleaved`` neighbours.  ``q_out`` may be
    q, ``k_out`` k.  Returns (q_out, k_out)."""
    if stream is not None:
        with torch.cuda.stream(_stream_obj(stream, (k if q is None else q).device)):
            return gdn_qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, axes,
                                    interleaved, q_out, k_out)
    return (_native or _binding()).qk_norm_rope(q, k, positions, inv_freq, axes, interleaved, eps,
                                                q_weight, k_weight, q_out, k_out)


def gdn_paged_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                     cu_seqlens: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                     positions: Optional[torch.Tensor] = None,
                     inv_freq: Optional[torch.Tensor] = None,
                     q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     axes: Optional[Sequence[int]] = None, interleaved: bool = False,
                     k_scale: Optional[torch.Tensor] = None,
                     v_scale: Optional[torch.Tensor] = None,
                     q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Appends new keys and values to a paged cache, keys normed and rotated
    on the way as by ``gdn_qk_norm_rope``, and the queries beside them (see
    ``gdn_paged_append`` in include/gdn_attention.h).  k, v: [T, Hkv, D], q:
    [T, Hq, D] or None, bf16 or fp32; k_cache, v_cache: [pages, page_size, Hkv,
    D] in their type, or float8_e4m3fn (for bf16) with k_scale, v_scale [Hkv]
    fp32, strided but for D; page_table: [N, max_pages] int32; seq_lens: [N]
    int32, the lengths with the new tokens; cu_seqlens: [N+1] int32, or None for
    T / N tokens of each sequence; positions: None for a token's index in its
    sequence.  Returns the queries, or None."""
    if stream is not None:
        with torch.cuda.stream(_stream_obj(stream, k.device)):
            return gdn_paged_append(k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens, q,
                                    positions, inv_freq, q_weight, k_weight, eps, axes,
                                    interleaved, k_scale, v_scale, q_out)
    return (_native or _binding()).paged_append(
        k, v, k_cache, v_cache, page_table, seq_lens, k_scale, v_scale, positions, inv_freq, axes,
        interleaved, eps, cu_seqlens, q, q_weight, k_weight, q_out)


def gdn_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        page_table: torch.Tensor, seq_lens: torch.Tensor,
                        scale: Optional[float] = None, gate: Optional[torch.Tensor] = None,
                        k_scale: Optional[torch.Tensor] = None,
                        v_scale: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        return_lse: bool = False, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """Attention of each sequence's newest tokens over its paged cache (see
    ``gdn_paged_attention`` in include/gdn_attention.h).  q: [N, Hq, D] (one
    token) or [N, L, Hq, D] (L up to 8, the last L of each sequence's tokens,
    each seeing those up to itself), bf16 or fp32; the cache as in
    ``gdn_paged_append``; scale: 1 / sqrt(D) by default; gate: like q, the
    output is multiplied by its sigmoid; ``out`` may be q or gate.  Returns out,
    or with ``lse`` or ``return_lse`` (out, lse [N, (L,) Hq] fp32).
    ``workspace`` is scratch of at least ``gdn_paged_attention_workspace_size``
    bytes, by default taken from the caching allocator for the call."""
    if stream is not None:
        with torch.cuda.stream(_stream_obj(stream, q.device)):
            return gdn_paged_attention(q, k_cache, v_cache, page_table, seq_lens, scale, gate,
                                       k_scale, v_scale, out, lse, return_lse, workspace)
    return (_native or _binding()).paged_attention(
        q, k_cache, v_cache, page_table, seq_lens, k_scale, v_scale, scale, gate, out, lse,
        return_lse, workspace)


def gdn_paged_attention_workspace_size(N: int, q_heads: int, kv_heads: int, head_dim: int,
                                       page_size: int, max_pages: int, new_tokens: int = 1,
                                       cache_dtype=torch.bfloat16) -> int:
    """Workspace bytes of ``gdn_paged_attention`` (0: none needed, or sizes
    that it does not support)."""
    dtype = GDN_F32 if cache_dtype == torch.float32 else GDN_BF16
    p = AttentionProblem(new_tokens=new_tokens, q_heads=q_heads, kv_heads=kv_heads,
                         head_dim=head_dim, dtype=dtype)
    c = PagedCache(dtype=_CACHE_DTYPES[cache_dtype], page_size=page_size, num_seqs=N,
                   max_pages=max_pages)
    return int(library().gdn_paged_attention_workspace_size(p, c))
