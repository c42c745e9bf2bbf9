"""The attention operators against plain 64-bit references: element by element,
within bounds that follow from the documented precision."""
import math
import random

import pytest
import torch

import gated_deltanet_linear_chunk_gb300 as gdn

import attention_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=BF16, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def frequencies(pairs, theta=1e4):
    return (theta ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / max(pairs, 1))).float()


def check(got, want, bound, what=""):
    got, ok, nan = got.double(), torch.isfinite(want), torch.isnan(want)
    others = int((torch.isnan(got) != nan).sum())
    assert others == 0, f"{what}: {others} NaN differ"
    others = int((got != want)[~ok & ~nan].sum())
    assert others == 0, f"{what}: {others} infinities differ"
    ratio = float(((got - want).abs() / bound.expand_as(want))[ok & (got != want)].amax()) \
        if bool((ok & (got != want)).any()) else 0.0
    assert ratio <= 1.0, f"{what}: off by {ratio} times the bound"


def inside(x, kind, g):
    """The same values as a slice of something wider: head by head beside
    gates, columns of a projection, or off 16-byte boundaries."""
    T, H, D = x.shape
    if kind == "gated":
        wide = normal(g, T, H, 2 * D, dtype=x.dtype)
        view = wide[..., :D]
    elif kind == "columns":
        wide = normal(g, T, H * D + 24, dtype=x.dtype)
        view = wide[:, 16:16 + H * D].unflatten(1, (H, D))
    elif kind == "odd":
        wide = normal(g, T, H * D + 3, dtype=x.dtype)
        view = wide[:, 1:1 + H * D].unflatten(1, (H, D))
    elif kind == "heads first":
        wide = normal(g, H, T, D, dtype=x.dtype)
        view = wide.transpose(0, 1)
    else:
        return x.contiguous()
    view.copy_(x)
    return view


ROPE = [  # dtype, T, Hq, Hk, D, pairs, norm, axes, interleaved, layout
    (BF16, 1, 24, 4, 256, 32, True, 1, False, "gated"),
    (BF16, 37, 24, 4, 256, 32, True, 1, False, "columns"),
    (BF16, 130, 8, 2, 128, 64, True, 3, False, "plain"),
    (BF16, 130, 8, 2, 128, 64, True, 3, True, "heads first"),
    (BF16, 9, 3, 1, 64, 32, False, 1, False, "odd"),
    (BF16, 9, 3, 1, 64, 32, True, 2, True, "odd"),
    (BF16, 700, 5, 5, 80, 20, True, 1, False, "plain"),      # words of 8, a half of 20: element by element
    (BF16, 11, 2, 1, 72, 0, True, 1, False, "plain"),
    (BF16, 5, 2, 1, 512, 256, True, 8, False, "plain"),
    (BF16, 3, 1, 0, 8, 4, True, 1, False, "plain"),
    (BF16, 3, 0, 2, 16, 8, True, 1, True, "plain"),
    (F32, 1, 9, 3, 74, 19, False, 1, True, "plain"),
    (F32, 33, 9, 3, 74, 19, True, 1, False, "odd"),
    (F32, 64, 4, 4, 128, 64, True, 1, False, "gated"),
    (F32, 64, 4, 1, 256, 16, True, 1, True, "columns"),
    (F32, 7, 2, 2, 512, 256, True, 3, False, "plain"),
    (F32, 7, 2, 2, 511, 255, True, 1, True, "plain"),
    (F32, 7, 2, 2, 1, 0, True, 1, False, "plain"),
    (F32, 5000, 2, 1, 2, 1, False, 1, False, "plain"),
]


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_norm_rope(case):
    dtype, T, Hq, Hk, D, pairs, norm, axes, interleaved, layout = case
    g = generator(T + D)
    f = frequencies(pairs) if pairs else None
    kw = dict(inv_freq=f, eps=EPS, interleaved=interleaved)
    pos = which = None
    if pairs:
        pos = torch.randint(0, 300000, (axes, T) if axes > 1 else (T,), generator=g,
                            device="cuda").to(torch.int32)
        which = [i % axes for i in range(pairs)] if axes > 1 else None
        kw.update(positions=pos, axes=which)
    x, w = [], []
    for H in (Hq, Hk):
        x.append(inside(normal(g, T, H, D, dtype=dtype, std=2.0), layout, g) if H else None)
        w.append(normal(g, D, dtype=F32, std=0.3, mean=1.0) if norm and H else None)
    got = gdn.gdn_qk_norm_rope(*x, q_weight=w[0], k_weight=w[1], **kw)
    for a, b, c in zip(x, w, got):
        if a is None:
            assert c is None
            continue
        y, err = ref.norm_rope(a, b, EPS, pos, f, which, interleaved)
        check(c, y, ref.rounded(y, err, dtype))
        assert c.is_contiguous() and c.dtype == dtype
    # In place, and into a strided result that is untouched between its heads.
    into = [None if a is None else inside(torch.zeros_like(a), "gated", g) for a in x]
    gdn.gdn_qk_norm_rope(*x, q_weight=w[0], k_weight=w[1], q_out=into[0], k_out=into[1], **kw)
    gdn.gdn_qk_norm_rope(*x, q_weight=w[0], k_weight=w[1], q_out=x[0], k_out=x[1], **kw)
    for a, b, c in zip(x, into, got):
        if a is not None:
            assert torch.equal(a, c) and torch.equal(b, c)


def test_rope_far_and_negative_positions():
    """Positions over the whole int32 range lose nothing: two radians per
    position at 2^31, where an angle in fp32 would be off by hundreds."""
    g = generator(1)
    pos = ints([0, 1, -1, 7, 10 ** 6, -10 ** 6, 2 ** 30 + 3, 2 ** 31 - 1, -2 ** 31])
    f = torch.tensor([2.0, 1.0, 0.7, 1e-3, 1e-7, 0.0, 6.2831855, 100.5], device="cuda")
    x = normal(g, 9, 2, 16, dtype=F32)
    got, _ = gdn.gdn_qk_norm_rope(x, positions=pos, inv_freq=f)
    y, err = ref.norm_rope(x, None, EPS, pos, f)
    check(got, y, ref.rounded(y, err, F32))


def test_rope_special_values_stay_in_their_rows_and_pairs():
    x = normal(generator(2), 6, 3, 64, dtype=F32)
    f = frequencies(16)
    f[3] = math.inf
    pos = ints(range(6))
    x[2, 1, 40] = math.nan  # not rotated: the head's norm spreads it
    x[4, 0, 5] = math.inf
    w = torch.ones(64, device="cuda")
    got, plain = gdn.gdn_qk_norm_rope(x, x, positions=pos, inv_freq=f, q_weight=w)
    bad = torch.isnan(got)
    assert bad[2, 1].all() and bad[..., [3, 19]].all()
    bad[2, 1] = bad[4, 0] = False
    bad[..., [3, 19]] = False
    assert not bad.any()
    bad = torch.isnan(plain)
    assert bad[2, 1, 40]
    bad[2, 1, 40] = bad[4, 0, 5] = bad[4, 0, 21] = False
    bad[..., [3, 19]] = False
    assert not bad.any()


# ---- the cache -------------------------------------------------------------------------------------------------


class Cache:
    """A paged cache for sequences of `lens` tokens at most: pages in random
    order, every place filled with `fill`, entries of the table that are not
    used out of range."""

    def __init__(self, g, lens, page_size, Hkv, D, dtype, order="heads", fill=None, spare=3):
        used = [-(-n // page_size) for n in lens]
        P = sum(used) + spare
        perm = torch.randperm(P, generator=g, device="cuda").tolist()
        width = max(used + [0]) + 1
        self.table, at = [], 0
        for u in used:
            self.table.append(perm[at:at + u] + [-1 - at] * (width - u))
            at += u
        shape = (P, Hkv, page_size, D) if order == "heads" else (P, page_size, Hkv, D)

        def make():
            x = normal(g, *shape, dtype=F32, std=30.0 if dtype == E4M3 else 1.0)
            if fill is not None:
                x.fill_(fill)
            x = x.to(dtype)
            return x.transpose(1, 2) if order == "heads" else x
        if order == "both":  # keys and values of a page together
            both = torch.empty(P, 2, page_size, Hkv, D, dtype=dtype, device="cuda")
            self.k, self.v = both[:, 0], both[:, 1]
            self.k.copy_(make())
            self.v.copy_(make())
        else:
            self.k, self.v = make(), make()
        self.scales = {}
        if dtype == E4M3:
            self.scales = {n: (torch.rand(Hkv, generator=g, device="cuda") + 0.5) / 30
                           for n in ("k_scale", "v_scale")}
        self.page_table = ints(self.table)

    def args(self, lens):
        return dict(k_cache=self.k, v_cache=self.v, page_table=self.page_table,
                    seq_lens=ints(lens), **self.scales)


def bits(x):
    return x.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


APPEND = [  # dtype, cache, new, lens, page, Hq, Hkv, D, pairs, norm, interleaved, order, layout
    (BF16, BF16, [1, 1, 1, 1], [1, 17, 16, 300], 16, 24, 4, 256, 32, True, False, "heads", "gated"),
    (BF16, BF16, [5, 0, 40, 1, 0], [5, 9, 77, 1, 0], 16, 6, 2, 128, 64, True, False, "tokens", "columns"),
    (BF16, BF16, [3, 33], [10, 33], 7, 0, 3, 64, 8, False, True, "both", "plain"),
    (BF16, BF16, [130], [130], 64, 3, 1, 64, 0, True, False, "heads", "odd"),
    (BF16, BF16, [9, 2], [9, 2], 1, 2, 2, 20, 5, True, False, "tokens", "odd"),
    (BF16, E4M3, [8, 8], [8, 500], 32, 8, 2, 128, 32, True, False, "heads", "gated"),
    (BF16, E4M3, [50, 1], [51, 1], 10, 0, 4, 64, 32, True, True, "tokens", "plain"),
    (BF16, E4M3, [5], [5], 4, 1, 1, 36, 9, True, False, "tokens", "odd"),
    (F32, F32, [20, 1, 0, 7], [30, 1, 4, 7], 10, 6, 2, 64, 32, False, True, "heads", "plain"),
    (F32, F32, [3, 3], [3, 40], 16, 4, 2, 256, 64, True, False, "both", "gated"),
]


@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(case):
    dtype, ct, new, lens, page, Hq, Hkv, D, pairs, norm, interleaved, order, layout = case
    g = generator(sum(lens) + D)
    c = Cache(g, lens, page, Hkv, D, ct, order)
    T = sum(new) + 3  # three tokens behind the last sequence
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    k, v = (inside(normal(g, T, Hkv, D, dtype=dtype), layout, g) for _ in range(2))
    q = inside(normal(g, T, Hq, D, dtype=dtype), layout, g) if Hq else None
    kw, qw = (normal(g, D, dtype=F32, std=0.3, mean=1.0) if norm else None for _ in range(2))
    f = frequencies(pairs) if pairs else None
    before = [bits(c.k).clone(), bits(c.v).clone()]
    mark = torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda") if Hq else None
    out = gdn.gdn_paged_append(k, v, cu_seqlens=ints(cu), q=q, inv_freq=f, q_weight=qw if Hq else None,
                               k_weight=kw, eps=EPS, interleaved=interleaved, q_out=mark,
                               **c.args(lens))
    stored, index = ref.places(cu, lens, c.table, page, c.k.shape[0], T)
    assert len(stored) == sum(new)
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    for t, j in index.items():
        pos[t] = j
    ky, ke = ref.norm_rope(k, kw, EPS, pos, f, None, interleaved)
    vy, ve = v.double(), torch.zeros_like(v.double())
    at = torch.tensor([[t, p, s] for t, p, s, _ in stored], device="cuda").t()
    for cache, y, e, scale, old in ((c.k, ky, ke, "k_scale", before[0]), (c.v, vy, ve, "v_scale", before[1])):
        y, e = y[at[0]], e[at[0]]
        if ct == E4M3:
            s = c.scales[scale].double()[:, None]
            y, e = (y / s).clamp(-448, 448), e / s + ref.U * (y / s).abs()
        now = bits(cache)
        check(now[at[1], at[2]].view(ct).float(), y, ref.rounded(y, e, ct))
        now = now.clone()
        now[at[1], at[2]] = old[at[1], at[2]]
        assert torch.equal(now, old)  # nothing else was touched
    if Hq:
        assert out is mark
        y, e = ref.norm_rope(q, qw, EPS, pos, f, None, interleaved)
        rows = torch.tensor(sorted(index), device="cuda", dtype=torch.int64)
        check(out[rows], y[rows], ref.rounded(y, e, dtype)[rows])
        assert (out[cu[-1]:] == 7.0).all()
    else:
        assert out is None


def test_append_leaves_out_what_has_no_place():
    """Pages out of range, lengths shorter than the new tokens, and tokens
    before the first sequence."""
    g = generator(5)
    c = Cache(g, [40, 40, 40], 8, 2, 64, BF16)
    P = c.k.shape[0]
    c.table[0][4], c.table[1][4] = P, -1
    c.table[2][0] = 2 ** 31 - 1
    c.page_table = ints(c.table)
    lens, cu = [40, 40, 3], [2, 14, 26, 31]
    k, v = normal(g, 31, 2, 64), normal(g, 31, 2, 64)
    q = normal(g, 31, 1, 64)
    before = c.k.clone()
    mark = torch.full_like(q, 7.0)
    gdn.gdn_paged_append(k, v, cu_seqlens=ints(cu), q=q, q_out=mark, **c.args(lens))
    stored, index = ref.places(cu, lens, c.table, 8, P, 31)
    assert len(stored) == 8 and len(index) == 29
    for t, p, s, _ in stored:
        assert torch.equal(c.k[p, s], k[t]) and torch.equal(c.v[p, s], v[t])
        before[p, s] = k[t]
    assert torch.equal(before, c.k)
    assert (mark[:2] == 7.0).all() and torch.equal(mark[2:], q[2:])


def test_append_by_equal_shares_with_positions_of_axes():
    """Without cu_seqlens every sequence has T / N new tokens; positions of
    several axes replace the indices."""
    g = generator(6)
    lens, L = [9, 3, 64], 3
    c = Cache(g, lens, 16, 2, 128, BF16)
    k, v, q = normal(g, 9, 2, 128), normal(g, 9, 2, 128), normal(g, 9, 6, 128)
    f, pos = frequencies(64), torch.randint(0, 4096, (3, 9), generator=g, device="cuda").to(torch.int32)
    axes = [i % 3 for i in range(64)]
    w = normal(g, 128, dtype=F32, std=0.3, mean=1.0)
    out = gdn.gdn_paged_append(k, v, q=q, positions=pos, inv_freq=f, axes=axes, q_weight=w,
                               k_weight=w, **c.args(lens))
    wq, wk = gdn.gdn_qk_norm_rope(q, k, positions=pos, inv_freq=f, axes=axes, q_weight=w, k_weight=w)
    assert torch.equal(out, wq)
    for t, p, s, _ in ref.places([0, 3, 6, 9], lens, c.table, 16, c.k.shape[0], 9)[0]:
        assert torch.equal(c.k[p, s], wk[t]) and torch.equal(c.v[p, s], v[t])


def test_append_to_8_bits_saturates():
    c = Cache(generator(7), [1], 1, 1, 64, E4M3)
    for s in c.scales.values():
        s.fill_(0.5)
    v = torch.linspace(-400, 400, 64, device="cuda").to(BF16).view(1, 1, 64)
    v[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 2.0 ** -11])
    gdn.gdn_paged_append(v, v, **c.args([1]))
    got = bits(c.v)[c.table[0][0], 0, 0].view(E4M3).float()
    want = (v[0, 0].float() / 0.5).clamp(-448, 448).to(E4M3).float()
    assert torch.equal(got[3:], want[3:]) and torch.isnan(got[2])
    assert got[0] == 448 and got[1] == -448


# ---- attention -------------------------------------------------------------------------------------------------

EDGES = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 300]
ATTENTION = [  # dtype, cache, lens, L, Hq, Hkv, D, page, gate, order
    (BF16, BF16, EDGES, 1, 24, 4, 256, 16, True, "heads"),
    (BF16, BF16, EDGES, 1, 6, 1, 128, 16, False, "tokens"),
    (BF16, BF16, EDGES, 3, 4, 2, 64, 10, True, "both"),
    (BF16, BF16, [5000], 1, 8, 1, 256, 16, False, "heads"),
    (BF16, BF16, [3, 2000, 1], 8, 6, 1, 256, 64, True, "heads"),
    (BF16, BF16, [700, 64], 8, 8, 1, 128, 7, True, "tokens"),
    (BF16, BF16, [700, 64], 5, 5, 1, 64, 1, False, "heads"),
    (BF16, BF16, [400, 7], 8, 16, 1, 128, 32, False, "heads"),   # 128 rows
    (BF16, BF16, [400, 7], 7, 33, 1, 64, 32, True, "both"),      # 231 rows
    (BF16, BF16, [900], 2, 16, 1, 256, 128, False, "heads"),
    (BF16, BF16, [900], 3, 16, 1, 256, 128, True, "heads"),
    (BF16, BF16, [90] * 200, 1, 3, 3, 64, 16, False, "heads"),   # more sequences than threads
    (BF16, BF16, [150, 40] * 80, 4, 24, 4, 64, 16, True, "heads"),  # narrow heads of many rows, a few pieces each
    (BF16, BF16, [300, 1, 77], 2, 16, 1, 64, 16, False, "tokens"),
    (BF16, E4M3, EDGES, 1, 16, 2, 128, 32, True, "heads"),
    (BF16, E4M3, EDGES, 2, 6, 3, 64, 10, False, "tokens"),
    (BF16, E4M3, [3000, 1, 0], 4, 6, 1, 256, 16, True, "heads"),
    (BF16, E4M3, [500, 8], 8, 9, 1, 128, 16, False, "both"),
    (F32, F32, EDGES, 1, 4, 2, 64, 16, True, "heads"),
    (F32, F32, EDGES, 3, 3, 1, 128, 10, False, "tokens"),
    (F32, F32, [2000, 1, 0, 9], 8, 6, 2, 256, 16, True, "both"),
    (F32, F32, [300], 1, 1, 1, 256, 300, False, "heads"),
    (F32, F32, [150, 40] * 80, 4, 24, 4, 64, 16, True, "heads"),
    (F32, F32, [500, 130, 64], 3, 4, 1, 64, 16, False, "tokens"),
]


def attend(q, c, lens, gate=None, **kw):
    """The call with statistics, its workspace full of NaN."""
    N, L = (q.shape[0], 1) if q.dim() == 3 else q.shape[:2]
    need = gdn.gdn_paged_attention_workspace_size(N, q.shape[-2], c.k.shape[2], q.shape[-1],
                                                  c.k.shape[1], c.page_table.shape[1], L, c.k.dtype)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    return gdn.gdn_paged_attention(q, gate=gate, return_lse=True, workspace=ws, **c.args(lens), **kw)


def check_attention(q, c, lens, got, gate=None, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    q4 = q if q.dim() == 4 else q[:, None]
    g4 = None if gate is None else gate.view(q4.shape) if q.dim() == 3 else gate
    out, err, lse, lse_err = ref.attention(q4, c.k, c.v, c.table, lens, scale, g4, **c.scales)
    check(got[0].view(q4.shape), out, ref.rounded(out, err, q.dtype), "out")
    check(got[1].view(q4.shape[:3]), lse, lse_err, "lse")


@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: str(c)[:100])
def test_attention(case):
    dtype, ct, lens, L, Hq, Hkv, D, page, gated, order = case
    g = generator(sum(lens) + L)
    lens = list(lens)
    random.Random(D).shuffle(lens)
    c = Cache(g, lens, page, Hkv, D, ct, order)
    q = normal(g, len(lens), L, Hq, D, dtype=dtype)
    gate = normal(g, len(lens), L, Hq, 2 * D, dtype=dtype)[..., D:] if gated else None
    if L == 1:
        q = q[:, 0]
        gate = gate[:, 0] if gated else None
    got = attend(q, c, lens, gate)
    check_attention(q, c, lens, got, gate)
    again = attend(q, c, lens, gate)
    assert torch.equal(bits(got[0]), bits(again[0])) and torch.equal(bits(got[1]), bits(again[1]))


@pytest.mark.parametrize("dtype,ct", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_attention_sees_nothing_else(dtype, ct):
    """NaN wherever a row does not look: places behind the lengths, other
    pages, and later ones of the new tokens, keys as well as values."""
    g = generator(11)
    lens, L, page = [40, 7, 130, 2, 0, 65], 4, 16
    clean = Cache(g, lens, page, 2, 128, ct)
    q = normal(g, len(lens), L, 6, 128, dtype=dtype)
    want = attend(q, clean, lens)
    dirty = Cache(g, lens, page, 2, 128, ct, fill=math.nan)
    dirty.table, dirty.page_table, dirty.scales = clean.table, clean.page_table, clean.scales
    for n, length in enumerate(lens):
        for j in range(length):
            p, s = clean.table[n][j // page], j % page
            bits_of = lambda x: x.view(torch.uint8) if ct == E4M3 else x  # noqa: E731
            bits_of(dirty.k)[p, s] = bits_of(clean.k)[p, s]
            bits_of(dirty.v)[p, s] = bits_of(clean.v)[p, s]
    got = attend(q, dirty, lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # The last token's key, then value, is NaN: only the last row knows.
    for cache in (dirty.k, dirty.v):
        for n, length in enumerate(lens):
            if length:
                j = length - 1
                at = cache[dirty.table[n][j // page]]
                (at.view(torch.uint8) if ct == E4M3 else at)[j % page] = 0x7F if ct == E4M3 else math.nan
        got = attend(q, dirty, lens)
        some = [n for n, length in enumerate(lens) if length]
        assert torch.equal(got[0][:, :L - 1], want[0][:, :L - 1])
        assert torch.equal(got[1][:, :L - 1], want[1][:, :L - 1])
        assert torch.isnan(got[0][some, L - 1]).all() and not torch.isnan(got[0][4]).any()


def test_attention_infinite_values_reach_those_that_see_them():
    g = generator(12)
    c = Cache(g, [50], 16, 1, 64, BF16)
    q = normal(g, 1, 3, 2, 64)
    j = 48  # seen by the last two rows
    c.v[c.table[0][j // 16], j % 16, 0, 5] = math.inf
    out, _ = attend(q, c, [50])
    assert torch.isfinite(out[0, 0]).all()
    assert (out[0, 1:, :, 5] == math.inf).all()
    out[0, 1:, :, 5] = 0.0
    assert torch.isfinite(out).all()


def test_attention_scores_of_minus_infinity():
    """Keys of -infinity count for nothing; a row that has no others is
    empty."""
    g = generator(13)
    c = Cache(g, [20, 20], 16, 1, 64, F32)
    q = torch.ones(2, 1, 64, device="cuda")
    c.k.fill_(0.25)
    for j in range(20):
        c.k[c.table[0][j // 16], j % 16] = -math.inf
        if j != 3:
            c.k[c.table[1][j // 16], j % 16] = -math.inf
    out, lse = attend(q, c, [20, 20])
    assert (out[0] == 0).all() and lse[0, 0] == -math.inf
    assert torch.allclose(out[1, 0], c.v[c.table[1][0], 3, 0], rtol=1e-6)


def test_attention_bad_pages_spoil_their_sequence_alone():
    g = generator(14)
    lens = [300, 300, 100]
    for ct, dtype in ((BF16, BF16), (E4M3, BF16), (F32, F32)):
        c = Cache(g, lens, 16, 2, 64, ct)
        q = normal(g, 3, 2, 4, 64, dtype=dtype)
        want = attend(q, c, lens)
        for bad in (c.k.shape[0], -1, 2 ** 31 - 1, -2 ** 31):
            table = [list(t) for t in c.table]
            table[1][7] = bad
            c.page_table = ints(table)
            got = attend(q, c, lens)
            assert torch.isnan(got[0][1]).all() and torch.isnan(got[1][1]).all()
            assert torch.equal(got[0][[0, 2]], want[0][[0, 2]])
            assert torch.equal(got[1][[0, 2]], want[1][[0, 2]])
        c.page_table = ints(c.table)


def test_attention_lengths_out_of_range_are_the_nearest():
    g = generator(15)
    c = Cache(g, [48, 48], 16, 1, 64, BF16)
    c.page_table = c.page_table[:, :3]
    q = normal(g, 2, 2, 64)
    want = attend(q, c, [48, 0])
    got = attend(q, c, [2 ** 31 - 1, -5])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("scale", [0.0, -0.7, 3.0])
def test_attention_scales(scale):
    g = generator(16)
    c = Cache(g, [200, 33], 16, 2, 64, BF16)
    q = normal(g, 2, 4, 64)
    check_attention(q, c, [200, 33], attend(q, c, [200, 33], scale=scale), scale=scale)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_steep_and_growing_scores(D):
    """Scores that grow along the sequence, by far more than the exponent's
    range in all, and one token that outweighs the rest."""
    g = generator(17)
    c = Cache(g, [1000], 16, 1, D, BF16)
    q = torch.zeros(1, 1, 2, D, dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    for j in range(1000):
        c.k[c.table[0][j // 16], j % 16, 0, 0] = j - 500.0
    check_attention(q, c, [1000], attend(q, c, [1000], scale=0.5), scale=0.5)
    q[..., 0] = -1.0
    check_attention(q, c, [1000], attend(q, c, [1000], scale=0.5), scale=0.5)


def test_attention_in_place_and_shared_pages():
    """out over q, out over gate, a table whose sequences share their first
    pages, and rows of a wider table."""
    g = generator(18)
    lens = [100, 80, 90]
    c = Cache(g, lens, 16, 2, 128, BF16)
    for n in (1, 2):
        c.table[n][:4] = c.table[0][:4]
    wide = torch.full((3, 40), -9, dtype=torch.int32, device="cuda")
    width = len(c.table[0])
    wide[:, 2:2 + width] = ints(c.table)
    c.page_table = wide[:, 2:2 + width]
    q = normal(g, 3, 2, 6, 256)[..., :128]
    gate = normal(g, 3, 2, 6, 128)
    got = attend(q, c, lens, gate)
    check_attention(q, c, lens, got, gate)
    a, b = q.clone(memory_format=torch.preserve_format), gate.clone()
    wide_q = normal(g, 3, 2, 6, 256)
    a = wide_q[..., :128]
    a.copy_(q)
    assert attend(a, c, lens, gate, out=a)[0] is a
    assert torch.equal(a, got[0])
    attend(q, c, lens, b, out=b)
    assert torch.equal(b, got[0])


def test_attention_past_32_bit_offsets():
    """A cache of more than 2^31 elements, its last pages used."""
    P, S, H, D = 2 ** 31 // (16 * 2 * 128) + 40, 16, 2, 128
    k = torch.empty(P, S, H, D, dtype=E4M3, device="cuda")
    v = torch.empty(P, S, H, D, dtype=E4M3, device="cuda")
    g = generator(19)

    class Big:
        pass
    c = Big()
    c.k, c.v, lens = k, v, [70, 33]
    c.table = [[P - 1, 3, P - 7, P // 2, 0], [P - 2, P - 3, 5, 6, 7]]
    c.page_table = ints(c.table)
    c.scales = dict(k_scale=torch.rand(H, generator=g, device="cuda"),
                    v_scale=torch.rand(H, generator=g, device="cuda"))
    c.args = lambda lens: dict(k_cache=k, v_cache=v, page_table=c.page_table, seq_lens=ints(lens),
                               **c.scales)
    x, y = normal(g, 103, H, D), normal(g, 103, H, D)
    gdn.gdn_paged_append(x, y, cu_seqlens=ints([0, 70, 103]), **c.args(lens))
    for t, p, s, _ in ref.places([0, 70, 103], lens, c.table, S, P, 103)[0][::9]:
        want = (x[t].float() / c.scales["k_scale"][:, None]).clamp(-448, 448).to(E4M3)
        assert torch.equal(k[p, s].view(torch.uint8), want.view(torch.uint8))
    q = normal(g, 2, 1, 4, D)
    check_attention(q, c, lens, attend(q, c, lens))


# ---- together --------------------------------------------------------------------------------------------------


class Layer:
    """Norms, rotation, cache and attention of one layer, token by token."""

    def __init__(self, dtype, ct, lens, room, L=1, seed=20):
        g = generator(seed)
        self.N, self.L, self.Hq, self.Hkv, self.D = len(lens), L, 6, 2, 128
        self.cache = Cache(g, [n + room for n in lens], 16, self.Hkv, self.D, ct)
        self.f = frequencies(16, 1e6)
        self.qw, self.kw = (normal(g, self.D, dtype=F32, std=0.3, mean=1.0) for _ in range(2))
        self.dtype, self.g = dtype, g
        self.lens = ints(lens)

    def tokens(self, T):
        return [normal(self.g, T, H, self.D, dtype=self.dtype) for H in (2 * self.Hq, self.Hkv, self.Hkv)]

    def append(self, q, k, v, cu=None):
        c = self.cache
        return gdn.gdn_paged_append(k, v, c.k, c.v, c.page_table, self.lens, cu_seqlens=cu, q=q,
                                    inv_freq=self.f, q_weight=self.qw, k_weight=self.kw, **c.scales)

    def step(self, qg, k, v):
        """L new tokens of each sequence: their outputs [N, L, Hq, D]."""
        c, Hq = self.cache, self.Hq
        self.lens.add_(self.L)
        q = self.append(qg[:, :Hq], k, v).view(self.N, self.L, Hq, self.D)
        gate = qg.view(self.N, self.L, 2 * Hq, self.D)[:, :, Hq:]
        return gdn.gdn_paged_attention(q, c.k, c.v, c.page_table, self.lens, gate=gate, **c.scales)


@pytest.mark.parametrize("dtype,ct", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
@pytest.mark.parametrize("L", [1, 4])
def test_prompt_and_tokens_together(dtype, ct, L):
    """A prompt appended at once and tokens appended one step at a time, each
    step's attention against the reference over what the cache then holds."""
    start = [5, 0, 33, 16]
    layer = Layer(dtype, ct, start, 4 * L, L)
    cu = ints([0, 5, 5, 38, 54])
    qg, k, v = layer.tokens(54)
    layer.append(qg[:, :6], k, v, cu)
    held = list(start)
    for _ in range(4):
        qg, k, v = layer.tokens(4 * L)
        out = layer.step(qg, k, v)
        held = [n + L for n in held]
        pos = torch.tensor([n - L + t for n in held for t in range(L)], device="cuda")
        q, err = ref.norm_rope(qg[:, :6], layer.qw, EPS, pos, layer.f)
        # The queries as they were rounded, from their own operator.
        rounded, _ = gdn.gdn_qk_norm_rope(qg[:, :6], positions=pos.to(torch.int32), inv_freq=layer.f,
                                          q_weight=layer.qw)
        check(rounded, q, ref.rounded(q, err, dtype))
        gate = qg.view(4, L, 12, 128)[:, :, 6:]
        want, bound, _, _ = ref.attention(rounded.view(4, L, 6, 128), layer.cache.k, layer.cache.v,
                                          layer.cache.table, held, 128 ** -0.5, gate,
                                          **layer.cache.scales)
        check(out, want, ref.rounded(want, bound, dtype))


def test_captured_steps_replay_with_new_lengths():
    """A step in a CUDA graph, replayed as the sequences grow over pages, gives
    what eager steps give; two graphs of one layer replayed on two streams
    share nothing but the cache."""
    eager, captured = Layer(BF16, BF16, [5, 120, 1], 40), Layer(BF16, BF16, [5, 120, 1], 40)
    inputs = [eager.tokens(3) for _ in range(20)]
    static = [x.clone() for x in inputs[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.step(*static)
        captured.lens.sub_(1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured.step(*static)
    for x in inputs:
        for a, b in zip(static, x):
            a.copy_(b)
        graph.replay()
        assert torch.equal(out, eager.step(*x))
    assert torch.equal(eager.cache.k, captured.cache.k)

    q = normal(generator(30), 3, 6, 128)
    c, graphs, outs = captured.cache, [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            o = gdn.gdn_paged_attention(q, c.k, c.v, c.page_table, captured.lens)
        graphs.append(gr)
        outs.append(o)
    want = gdn.gdn_paged_attention(q, c.k, c.v, c.page_table, captured.lens)
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_captured_behind_copies_and_events():
    """The launches follow a copy, and another stream's work, in a captured
    graph as they follow a kernel."""
    layer = Layer(BF16, BF16, [64, 200, 3], 10)
    qg, k, v = layer.tokens(3)
    layer.lens.add_(1)
    c, q = layer.cache, qg[:, :6]
    want_q = layer.append(q, k, v)
    want = gdn.gdn_paged_attention(want_q, c.k, c.v, c.page_table, layer.lens)
    hold_k, hold_lens = torch.zeros_like(k), torch.zeros_like(layer.lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hold_k.copy_(k)  # copies: contiguous tensors
        got_q = gdn.gdn_paged_append(hold_k, v, c.k, c.v, c.page_table, layer.lens, q=q,
                                     inv_freq=layer.f, q_weight=layer.qw, k_weight=layer.kw)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            hold_lens.copy_(layer.lens)
            a = gdn.gdn_paged_attention(got_q, c.k, c.v, c.page_table, hold_lens)
        b = gdn.gdn_paged_attention(got_q, c.k, c.v, c.page_table, layer.lens)
        torch.cuda.current_stream().wait_stream(side)
        r, _ = gdn.gdn_qk_norm_rope(a, q_weight=layer.qw)
    for _ in range(5):
        hold_lens.zero_()
        hold_k.zero_()
        c.k.zero_()
        layer.append(q, k, v)
        prefix = c.k.clone()
        graph.replay()
        assert torch.equal(got_q, want_q) and torch.equal(c.k, prefix)
        assert torch.equal(a, b)
        assert torch.equal(r, gdn.gdn_qk_norm_rope(b, q_weight=layer.qw)[0])
    assert want.shape == a.shape


def test_calls_from_host_threads():
    """Calls from several host threads, each on a stream of its own."""
    import threading
    layer = Layer(BF16, BF16, [500, 64, 1, 900], 4)
    c = layer.cache
    qs = [normal(generator(40 + i), 4, 6, 128) for i in range(4)]
    want = [gdn.gdn_paged_attention(q, c.k, c.v, c.page_table, layer.lens) for q in qs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                out = gdn.gdn_paged_attention(qs[i], c.k, c.v, c.page_table, layer.lens)
                s.synchronize()
                if not torch.equal(out, want[i]):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_calls_on_a_stream():
    """`stream=` runs the call there, after what was put on it before."""
    layer = Layer(BF16, BF16, [64, 200], 10)
    qg, k, v = layer.tokens(2)
    c, s = layer.cache, torch.cuda.Stream()
    layer.lens.add_(1)
    torch.cuda.synchronize()
    q = gdn.gdn_paged_append(k, v, c.k, c.v, c.page_table, layer.lens, q=qg[:, :6], stream=s)
    out = gdn.gdn_paged_attention(q, c.k, c.v, c.page_table, layer.lens, stream=s)
    r, _ = gdn.gdn_qk_norm_rope(q, q_weight=layer.qw, stream=s)
    s.synchronize()
    want = gdn.gdn_paged_attention(q, c.k, c.v, c.page_table, layer.lens)
    assert torch.equal(out, want)
    assert torch.equal(r, gdn.gdn_qk_norm_rope(q, q_weight=layer.qw)[0])


def test_nothing_to_do():
    g = generator(21)
    c = Cache(g, [5, 0], 16, 2, 64, BF16)
    none = torch.zeros(0, 2, 64, dtype=BF16, device="cuda")
    before = c.k.clone()
    q, k = gdn.gdn_qk_norm_rope(none, none, q_weight=torch.ones(64, device="cuda"))
    assert q.shape == k.shape == (0, 2, 64)
    assert gdn.gdn_paged_append(none, none, cu_seqlens=ints([0, 0, 0]), **c.args([5, 0])) is None
    assert torch.equal(before, c.k)
    args = c.args([5, 0])
    args["page_table"], args["seq_lens"] = args["page_table"][:0], args["seq_lens"][:0]
    assert gdn.gdn_paged_attention(none, **args).shape == (0, 2, 64)
    # No room at all: every sequence is empty.
    args = c.args([5, 0])
    args["page_table"] = args["page_table"][:, :0]
    out, lse = gdn.gdn_paged_attention(normal(g, 2, 4, 64), return_lse=True, **args)
    assert (out == 0).all() and (lse == -math.inf).all()
