"""Every variant of the paged attention's kernels that a call can reach: element
types, head widths, rows per key head, page sizes that do and do not let 16 tokens
share a page, rows on and off 16-byte boundaries; what a score or a value can be in
each of the three cache types; and sequences long enough for many pieces, with
answers that are exact."""
import math

import pytest
import torch

import gated_deltanet_linear_chunk_gb300 as gdn

import attention_ref as ref
from test_attention_ops_gpu import (BF16, E4M3, F32, Cache, Layer, attend, bits, check_attention, generator, inside,
                                    ints, normal)

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (BF16, BF16), "e4m3": (BF16, E4M3), "f32": (F32, F32)}
# New tokens and query heads per key head, for each number of rows that a kernel
# takes: those of the tensor cores, and those in fp32.
ROWS = {8: (1, 8), 7: (7, 1), 16: (2, 8), 24: (4, 6), 32: (4, 8), 48: (8, 6), 64: (8, 8), 80: (8, 10)}
ROWS_F32 = {1: (1, 1), 4: (2, 2), 8: (8, 1), 16: (2, 8), 24: (4, 6)}
VARIANTS = [(name, D, rows) for name in TYPES for D in (64, 128, 256)
            for rows in (ROWS_F32 if name == "f32" else ROWS)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def put(cache, table, j, columns, value):
    """`value` at some columns of the cache's token j, in every head."""
    S = cache.shape[1]
    at = (cache.view(torch.uint8) if cache.dtype == E4M3 else cache)[table[j // S], j % S]
    one = torch.tensor([value], dtype=F32).to(cache.dtype)
    at[..., columns] = (one.view(torch.uint8) if cache.dtype == E4M3 else one).item()


@pytest.mark.parametrize("name,D,rows", VARIANTS, ids=lambda v: str(v))
@pytest.mark.parametrize("page", [16, 10])
def test_variant(name, D, rows, page):
    """A few lengths about the tiles' sizes, gated; pages of 10 with all rows of
    queries, gates and results off 16-byte boundaries.  The newest values of
    some sequences are not finite in a column, which the rows that see them show
    and no others."""
    dtype, ct = TYPES[name]
    L, G = (ROWS_F32 if name == "f32" else ROWS)[rows]
    g = generator(D + rows + page)
    lens, Hkv = [65, 0, 300, 1, 63, 64, 300], 2
    N = len(lens)
    c = Cache(g, lens, page, Hkv, D, ct, "heads" if page == 16 else "tokens")
    put(c.v, c.table[2], 299, 3, math.nan)
    if ct != E4M3:
        put(c.v, c.table[5], 63, 7, math.inf)
    odd = page == 10
    q, gate, out = (inside(normal(g, N * L, Hkv * G, D, dtype=dtype), "odd" if odd else "plain", g)
                    .unflatten(0, (N, L)) for _ in range(3))
    assert (q.data_ptr() % 16 != 0) == odd
    got = attend(q, c, lens, gate, out=out)
    assert got[0] is out
    check_attention(q, c, lens, got, gate)
    plain = attend(q.contiguous(), c, lens, gate.contiguous())
    assert torch.equal(bits(plain[0]), bits(got[0])) and torch.equal(bits(plain[1]), bits(got[1]))


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("odd", ["q", "gate", "out"])
def test_one_tensor_off_its_words(name, odd):
    """Queries, gates or results alone off 16-byte boundaries, nothing beside the
    results written."""
    dtype, ct = TYPES[name]
    g = generator(3)
    lens = [100, 17]
    c = Cache(g, lens, 16, 2, 64, ct)
    x = {n: normal(g, 2, 6, 64, dtype=dtype) for n in ("q", "gate", "out")}
    want = attend(x["q"], c, lens, x["gate"])
    wide = torch.full((2, 6 * 64 + 3), 7.0, dtype=dtype, device="cuda")
    view = wide[:, 1:1 + 6 * 64].unflatten(1, (6, 64))
    view.copy_(x[odd])
    x[odd] = view
    got = attend(x["q"], c, lens, x["gate"], out=x["out"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (wide[:, 0] == 7.0).all() and (wide[:, -2:] == 7.0).all()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("L,G", [(1, 4), (4, 8)])
@pytest.mark.parametrize("scale", [0.0, -0.7, 3.0])
def test_scales(name, L, G, scale):
    dtype, ct = TYPES[name]
    g = generator(16)
    lens = [200, 33]
    c = Cache(g, lens, 16, 2, 64, ct)
    q = normal(g, 2, L, 2 * G, 64, dtype=dtype)
    check_attention(q, c, lens, attend(q, c, lens, scale=scale), scale=scale)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("L,G", [(1, 2), (4, 8)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_that_grow_by_far_more_than_the_exponents_range(name, L, G, D, sign):
    """One column of the keys counts up; queries pick it with either sign, so that
    scores grow or fall along the sequence."""
    dtype, ct = TYPES[name]
    g = generator(17)
    length = 900
    c = Cache(g, [length], 16, 1, D, ct)
    q = torch.zeros(1, L, G, D, dtype=dtype, device="cuda")
    q[..., 0] = sign
    steps = torch.arange(length, device="cuda", dtype=F32) - 450.0
    if ct == E4M3:
        c.scales["k_scale"] = torch.full((1,), 2.0, device="cuda")
        steps = steps / 2
    at = torch.tensor([[c.table[0][j // 16], j % 16] for j in range(length)], device="cuda").t()
    if ct == E4M3:
        c.k.view(torch.uint8)[at[0], at[1], 0, 0] = steps.to(ct).view(torch.uint8)
    else:
        c.k[at[0], at[1], 0, 0] = steps.to(ct)
    check_attention(q, c, [length], attend(q, c, [length], scale=0.5), scale=0.5)


@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("L,G", [(1, 4), (4, 8)])
def test_scores_of_minus_infinity(name, L, G):
    """Keys of -infinity, which an 8-bit cache has none of, count for nothing; a
    row that has no others is empty."""
    dtype, ct = TYPES[name]
    g = generator(13)
    lens = [150, 150]
    c = Cache(g, lens, 16, 1, 64, ct)
    q = torch.ones(2, L, G, 64, dtype=dtype, device="cuda")
    for j in range(150):
        put(c.k, c.table[0], j, slice(None), -math.inf)
        put(c.k, c.table[1], j, slice(None), 0.25 if j == 77 else -math.inf)
    out, lse = attend(q, c, lens)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    token = c.v[c.table[1][77 // 16], 77 % 16, 0]
    assert torch.equal(out[1], token.expand(L, G, 64))
    assert float((lse[1] - 2.0).abs().max()) <= 16 * ref.U * 2.0


@pytest.mark.parametrize("name", TYPES)
def test_queries_of_minus_infinity(name):
    """Queries of -infinity in one column against keys that are positive there but
    for one token's: a score of +infinity beside those of -infinity is NaN."""
    dtype, ct = TYPES[name]
    c = Cache(generator(4), [40], 16, 1, 64, ct)
    q = torch.zeros(1, 3, 64, dtype=dtype, device="cuda")
    for j in range(40):
        put(c.k, c.table[0], j, 5, 1.0)
    q[0, 1, 5] = -math.inf
    out, lse = attend(q, c, [40])
    assert (out[0, 1] == 0).all() and lse[0, 1] == -math.inf
    assert torch.isfinite(out[0, [0, 2]]).all()
    put(c.k, c.table[0], 20, 5, -1.0)
    out, lse = attend(q, c, [40])
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    assert torch.isfinite(out[0, [0, 2]]).all()


# ---- every token once ------------------------------------------------------------------------------------------


@pytest.mark.parametrize("name,D,rows", [v for v in VARIANTS if v[2] in (1, 8, 16, 24, 48, 64)], ids=lambda v: str(v))
def test_every_token_counts_once(name, D, rows):
    """Queries of zero, so that every weight is one, and values of one in column
    j % D of token j (of the second head, j / 7 % D), zero elsewhere: a column's
    result is the number of its tokens over the length, exact but for its last
    rounding, and the log-sum-exp the length's logarithm.  The lengths give at most
    61 tokens a column, so that one too many or too few shows."""
    dtype, ct = TYPES[name]
    L, G = (ROWS_F32 if name == "f32" else ROWS)[rows]
    lens, Hkv, page = [60 * D + 37, 17 * D + 1, 1, 5 * D, 3, D - 1, 29 * D + 63], 2, 16
    N = len(lens)
    g = generator(D + rows)
    c = Cache(g, lens, page, Hkv, D, ct)
    for s in c.scales:
        c.scales[s] = torch.ones(Hkv, device="cuda")
    one = torch.eye(D, device="cuda").to(ct)
    as_bytes = (lambda x: x.view(torch.uint8)) if ct == E4M3 else (lambda x: x)
    for n, length in enumerate(lens):
        j = torch.arange(length, device="cuda")
        pages = ints(c.table[n]).long()[j // page]
        for h, column in enumerate((j % D, j // 7 % D)):
            as_bytes(c.v)[pages, j % page, h] = as_bytes(one)[column]
    q = torch.zeros(N, L, Hkv * G, D, dtype=dtype, device="cuda")
    out, lse = attend(q, c, lens)
    step = ref.HALF_STEP[dtype] + 16 * ref.U
    for n, length in enumerate(lens):
        for t in range(L):
            seen = length - L + 1 + t
            if seen <= 0:
                assert (out[n, t] == 0).all() and (lse[n, t] == -math.inf).all()
                continue
            j = torch.arange(seen, device="cuda")
            counts = torch.stack([torch.bincount(x, minlength=D) for x in (j % D, j // 7 % D)])
            counts = counts.repeat_interleave(G, 0).double()
            assert bool(((out[n, t].double() * seen - counts).abs() <= step * counts).all()), (n, t)
            z = math.log(seen)
            # log2 and its sum with the maximum, and ln 2: a few steps of log(seen) + 7
            assert float((lse[n, t].double() - z).abs().max()) <= 8 * ref.U * (z + 7), (n, t)


# ---- one after the other ---------------------------------------------------------------------------------------


def test_attention_waits_for_what_it_reads_in_a_graph():
    """In a captured graph the attention follows the append, a copy and another
    stream's work: everything that it reads is spoilt before each replay, and the
    results are those of calls with the device synchronised between them."""
    layer = Layer(BF16, BF16, [64, 200, 3], 10)
    qg, k, v = layer.tokens(3)
    layer.lens.add_(1)
    c, q = layer.cache, qg[:, :6]
    clean = c.k.clone(), c.v.clone()
    want_q = layer.append(q, k, v)
    torch.cuda.synchronize()
    want = gdn.gdn_paged_attention(want_q, c.k, c.v, c.page_table, layer.lens)
    torch.cuda.synchronize()
    want_r, _ = gdn.gdn_qk_norm_rope(want, q_weight=layer.qw)
    held = c.k.clone(), c.v.clone()
    assert not torch.equal(held[0], clean[0]) and not torch.equal(held[1], clean[1])
    hold_k, hold_lens = torch.zeros_like(k), torch.zeros_like(layer.lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hold_k.copy_(k)
        got_q = gdn.gdn_paged_append(hold_k, v, c.k, c.v, c.page_table, layer.lens, q=q,
                                     inv_freq=layer.f, q_weight=layer.qw, k_weight=layer.kw)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            hold_lens.copy_(layer.lens)
            a = gdn.gdn_paged_attention(got_q, c.k, c.v, c.page_table, hold_lens)
        b = gdn.gdn_paged_attention(got_q, c.k, c.v, c.page_table, layer.lens)
        torch.cuda.current_stream().wait_stream(side)
        r, _ = gdn.gdn_qk_norm_rope(a, q_weight=layer.qw)
    for _ in range(10):
        for n, length in enumerate(layer.lens.tolist()):  # the new tokens' places
            for cache in (c.k, c.v):
                cache[c.table[n][(length - 1) // 16], (length - 1) % 16] = 3.0
        for x in (hold_k, hold_lens, got_q, a, b, r):
            x.fill_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got_q, want_q)
        assert torch.equal(c.k, held[0]) and torch.equal(c.v, held[1])
        assert torch.equal(a, want) and torch.equal(b, want) and torch.equal(r, want_r)


@pytest.mark.parametrize("name", TYPES)
def test_calls_one_after_the_other_share_a_workspace(name):
    """Calls of one stream, none waited for, with one workspace between them."""
    dtype, ct = TYPES[name]
    g = generator(9)
    lens = [900, 1, 333, 64]
    c = Cache(g, lens, 16, 2, 128, ct)
    args = c.args(lens)
    qs = [normal(g, 4, 2, 12, 128, dtype=dtype) for _ in range(8)]
    want = [gdn.gdn_paged_attention(q, **args) for q in qs]
    need = gdn.gdn_paged_attention_workspace_size(4, 12, 2, 128, 16, c.page_table.shape[1], 2, ct)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = [gdn.gdn_paged_attention(q, workspace=ws, **args) for _ in range(4) for q in qs]
    for i, y in enumerate(got):
        assert torch.equal(bits(y), bits(want[i % 8]))
