"""The attention operators' C ABI and binding without a GPU: bad arguments are
refused before anything is launched."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_chunk_gb300 as gdn
from gated_deltanet_linear_chunk_gb300.attention import AttentionProblem, PagedCache, RopeProblem

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)
A = 0x10000000  # an aligned fake device address; never dereferenced here
STEP = 0x1000000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return gdn.library()


def at(i):
    return A + i * STEP


def rope_problem(T=10, Hq=4, Hk=2, D=64, dtype=0, R=32, axes=1, axis=None, eps=1e-6, **kw):
    p = RopeProblem(total_tokens=T, q_heads=Hq, kv_heads=Hk, head_dim=D, dtype=dtype, rotary_dim=R,
                    num_axes=axes, eps=eps, axis_stride=T)
    for name, heads in (("q", Hq), ("k", Hk), ("v", Hk), ("q_out", Hq), ("k_out", Hk)):
        setattr(p, name + "_stride", heads * D)
        setattr(p, name + "_head_stride", D)
    if axis is not None:
        p.freq_axis = (ctypes.c_uint8 * len(axis))(*axis)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def rope(lib, p, q=at(0), k=at(1), qw=None, kw=None, pos=at(2), f=at(3), qo=at(4), ko=at(5)):
    return lib.gdn_qk_norm_rope(p, q, k, qw, kw, pos, f, qo, ko, None)


def test_rope_refusals(lib):
    assert rope(lib, None) == INVALID
    for kw in (dict(T=-1), dict(T=BIG), dict(Hq=-1), dict(Hk=-1), dict(Hq=5000), dict(D=0),
               dict(R=-2), dict(R=66), dict(axes=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(axes=2, axis=[2] * 16), dict(axes=2, axis=[0] * 16, axis_stride=9),
               dict(q_stride=255), dict(q_head_stride=63), dict(k_out_stride=127),
               dict(q_out_head_stride=0)):
        assert rope(lib, rope_problem(**kw)) == INVALID, kw
    for kw in (dict(D=513, R=2), dict(R=31), dict(axes=9), dict(dtype=2), dict(dtype=3)):
        assert rope(lib, rope_problem(**kw)) == UNSUPPORTED, kw
    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None),
               dict(f=None), dict(qo=at(1)), dict(ko=at(0)), dict(ko=at(4))):
        assert rope(lib, rope_problem(), **kw) == INVALID, kw
    assert rope(lib, rope_problem(q_out_stride=512), qo=at(0)) == INVALID  # in place, other rows
    assert rope(lib, rope_problem(R=0)) == INVALID                         # angles without rotation
    assert rope(lib, rope_problem(Hq=0)) == INVALID                        # queries of no heads
    assert rope(lib, rope_problem(Hq=0), q=None, qo=None, qw=at(6)) == INVALID
    for kw in (dict(q=A + 1), dict(ko=at(5) + 1), dict(pos=at(2) + 2), dict(f=at(3) + 1),
               dict(qw=at(6) + 2), dict(kw=at(6) + 2)):
        assert rope(lib, rope_problem(), **kw) == MISALIGNED, kw
    assert rope(lib, rope_problem(T=0)) == OK
    assert rope(lib, rope_problem(Hq=0, Hk=0), q=None, k=None, qo=None, ko=None) == OK


def cache(dtype=0, N=3, P=20, S=16, H=2, D=64, width=5, scales=False, **kw):
    c = PagedCache(k=at(8), v=at(9), dtype=dtype, num_pages=P, page_size=S, num_seqs=N,
                   max_pages=width, page_table=at(10), table_stride=width, seq_lens=at(11))
    for name in ("k", "v"):
        setattr(c, name + "_page_stride", S * H * D)
        setattr(c, name + "_token_stride", H * D)
        setattr(c, name + "_head_stride", D)
    if scales:
        c.k_scale, c.v_scale = at(12), at(13)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = (dict(N=-1), dict(P=-1), dict(P=0), dict(P=1 << 31), dict(S=0), dict(S=(1 << 20) + 1),
              dict(width=-1), dict(width=1 << 28), dict(table_stride=4), dict(page_table=None),
              dict(seq_lens=None), dict(k=None), dict(v=None), dict(scales=True),
              dict(dtype=3), dict(dtype=3, scales=True, k_scale=None), dict(k_page_stride=2047),
              dict(k_token_stride=127), dict(k_head_stride=63), dict(v_page_stride=0),
              dict(k_page_stride=1 << 62))


def append(lib, p, c, q=at(0), k=at(1), v=at(2), qw=None, kw=None, pos=None, f=at(3), cu=at(5),
           qo=at(4)):
    return lib.gdn_paged_append(p, c, q, k, v, qw, kw, pos, f, cu, qo, None)


def test_append_refusals(lib):
    assert append(lib, None, cache()) == INVALID
    assert append(lib, rope_problem(), None) == INVALID
    for kw in BAD_CACHES:
        assert append(lib, rope_problem(), cache(**kw)) == INVALID, kw
    for kw in (dict(dtype=1), dict(dtype=2)):
        assert append(lib, rope_problem(), cache(**kw)) == UNSUPPORTED, kw
    assert append(lib, rope_problem(dtype=1), cache(dtype=3, scales=True)) == UNSUPPORTED
    for kw in (dict(Hk=0), dict(T=-1), dict(k_stride=1), dict(v_head_stride=1),
               dict(axes=2, axis=[0] * 16)):
        assert append(lib, rope_problem(**kw), cache(H=kw.get("Hk", 2) or 2)) == INVALID, kw
    for kw in (dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(f=None), dict(qo=at(1)),
               dict(qo=at(2)), dict(qo=at(8)), dict(k=at(8)), dict(v=at(9)),
               dict(cu=None)):  # 10 tokens of 3 sequences
        assert append(lib, rope_problem(), cache(), **kw) == INVALID, kw
    assert append(lib, rope_problem(), cache(v=at(8))) == INVALID
    assert append(lib, rope_problem(), cache(N=0), cu=None) == INVALID
    for kw in (dict(k=at(1) + 1), dict(cu=at(5) + 2), dict(pos=at(6) + 2)):
        assert append(lib, rope_problem(), cache(), **kw) == MISALIGNED, kw
    for kw in (dict(k=at(8) + 1), dict(page_table=at(10) + 2), dict(seq_lens=at(11) + 1),
               dict(dtype=3, scales=True, v_scale=at(13) + 2)):
        assert append(lib, rope_problem(), cache(**kw)) == MISALIGNED, kw
    assert append(lib, rope_problem(T=0), cache()) == OK
    assert append(lib, rope_problem(T=0), cache(N=0)) == OK


def attention_problem(L=1, Hq=4, Hkv=2, D=64, dtype=0, ws=at(14), wsb=BIG, **kw):
    p = AttentionProblem(new_tokens=L, q_heads=Hq, kv_heads=Hkv, head_dim=D, dtype=dtype, scale=0.1,
                         workspace=ws, workspace_bytes=wsb)
    for name in ("q", "gate", "out"):
        setattr(p, name + "_stride", Hq * D)
        setattr(p, name + "_head_stride", D)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def attend(lib, p, c, q=at(0), gate=None, out=at(1), lse=None):
    return lib.gdn_paged_attention(p, c, q, gate, out, lse, None)


def test_attention_refusals(lib):
    assert attend(lib, None, cache()) == INVALID
    assert attend(lib, attention_problem(), None) == INVALID
    for kw in BAD_CACHES:
        assert attend(lib, attention_problem(), cache(**kw)) == INVALID, kw
    assert attend(lib, attention_problem(L=8, Hq=4096, Hkv=4096, q_stride=1 << 20), cache(N=1 << 17)) == INVALID
    for kw in (dict(L=0), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(Hq=8192), dict(q_stride=255),
               dict(q_head_stride=63), dict(out_stride=255)):
        assert attend(lib, attention_problem(**kw), cache()) == INVALID, kw
    for kw in (dict(L=9), dict(Hq=5), dict(D=96), dict(D=32), dict(dtype=2), dict(dtype=3)):
        assert attend(lib, attention_problem(**kw), cache()) == UNSUPPORTED, kw
    assert attend(lib, attention_problem(), cache(dtype=1)) == UNSUPPORTED
    assert attend(lib, attention_problem(dtype=1), cache(dtype=3, scales=True)) == UNSUPPORTED
    for kw in (dict(q=None), dict(out=None), dict(out=at(8)), dict(out=at(9)), dict(lse=at(0)),
               dict(lse=at(1)), dict(lse=at(8)), dict(gate=at(2), lse=at(2))):
        assert attend(lib, attention_problem(), cache(), **kw) == INVALID, kw
    assert attend(lib, attention_problem(out_stride=512), cache(), out=at(0)) == INVALID
    assert attend(lib, attention_problem(gate_stride=512), cache(), gate=at(1)) == INVALID
    assert attend(lib, attention_problem(gate_stride=1), cache(), gate=at(2)) == INVALID
    for kw in (dict(q=at(0) + 1), dict(out=at(1) + 1), dict(gate=at(2) + 1), dict(lse=at(3) + 2)):
        assert attend(lib, attention_problem(), cache(), **kw) == MISALIGNED, kw
    # rows of the cache off 16-byte boundaries
    for kw in (dict(k=at(8) + 2), dict(v=at(9) + 8), dict(k_token_stride=132, k_page_stride=4096),
               dict(v_head_stride=68, v_token_stride=256, v_page_stride=8192),
               dict(k_page_stride=2052)):
        assert attend(lib, attention_problem(), cache(**kw)) == MISALIGNED, kw
    assert attend(lib, attention_problem(), cache(N=0)) == OK


def test_attention_workspace(lib):
    size = lib.gdn_paged_attention_workspace_size
    assert size(None, cache()) == 0 and size(attention_problem(), None) == 0
    assert size(attention_problem(D=96), cache()) == 0
    assert size(attention_problem(), cache(width=1 << 28)) == 0
    assert size(attention_problem(), cache(N=0)) == 0
    c = cache(width=500)
    need = size(attention_problem(), c)
    assert need > 0
    assert need == gdn.gdn_paged_attention_workspace_size(3, 4, 2, 64, 16, 500)
    for ws, wsb in ((None, 0), (at(14), need - 1), (at(14) + 8, need)):
        assert attend(lib, attention_problem(ws=ws, wsb=wsb), c) == WORKSPACE


def tensors(dtype=torch.bfloat16, N=2, P=4, S=16, H=2, D=64):
    kc = torch.zeros(P, S, H, D, dtype=dtype)
    return dict(k_cache=kc, v_cache=kc.clone(), page_table=torch.zeros(N, 3, dtype=torch.int32),
                seq_lens=torch.ones(N, dtype=torch.int32))


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    bf = torch.bfloat16
    q, k = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(2, 2, 64, dtype=bf)
    with pytest.raises(ValueError, match="one CUDA device"):
        gdn.gdn_qk_norm_rope(q, k)
    with pytest.raises(ValueError, match="one CUDA device"):
        gdn.gdn_paged_append(k, k.clone(), **tensors())
    with pytest.raises(ValueError, match="one CUDA device"):
        gdn.gdn_paged_attention(q, **tensors())
    with pytest.raises(ValueError, match="must be given"):
        gdn.gdn_qk_norm_rope(None)
    for bad in (q.half(), q.double()):
        with pytest.raises(TypeError):
            gdn.gdn_qk_norm_rope(bad)
        with pytest.raises(TypeError):
            gdn.gdn_paged_attention(bad, **tensors())
    with pytest.raises(ValueError, match="contiguous within its heads"):
        gdn.gdn_qk_norm_rope(torch.zeros(2, 64, 4, dtype=bf).transpose(1, 2))
    with pytest.raises(ValueError, match="dimensions"):
        gdn.gdn_qk_norm_rope(q[0])
    with pytest.raises(ValueError, match="dimensions"):
        gdn.gdn_paged_attention(q[0], **tensors())
    with pytest.raises(TypeError, match="must be a tensor"):
        gdn.gdn_paged_attention([1.0], **tensors())
