"""What softmax weights lose on their way into the products, against 64 bits and
closer than a rounding to 16 bits would allow."""
import math

import pytest
import torch

import attention_ref as ref
from test_attention_ops_gpu import BF16, E4M3, F32, Cache, attend, check, generator, normal

pytestmark = pytest.mark.gpu

U = ref.U


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def exact(q, c, n, length, scale, part):
    """(out, bound before the last rounding) of q [rows, D], all of which see the
    `length` tokens of sequence n of a cache with one key head.  `part`: what a
    weight in the products is off by, of itself."""
    S = c.k.shape[1]
    held = torch.tensor(c.table[n][:-(-length // S)], device="cuda")

    def rows(cache, by):
        x = cache.view(torch.uint8)[held].view(cache.dtype) if by else cache[held]
        x = x.flatten(0, 1)[:length, 0].double()
        return x * c.scales[by].double() if by else x
    eight = c.k.dtype == E4M3
    k, v = rows(c.k, "k_scale" if eight else None), rows(c.v, "v_scale" if eight else None)
    x, D = q.double(), q.shape[-1]
    s, mag = scale * x @ k.t(), abs(scale) * x.abs() @ k.abs().t()
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    # As in attention_ref: a score's products and sum, the exponent's roundings,
    # ex2, a factor per tile at most, the sums of the tokens.
    es = (2 * D + 8) * U * mag
    if eight:
        es = es + 2.0 ** -24 * abs(scale) * x.abs().amax(-1, keepdim=True) * k.abs().sum(-1)
    rel = (es + 6 * U * (s.abs() + m.abs())).amax(-1, keepdim=True) + (8 + 3 * length) * U
    weighted = (p @ v.abs()) / l
    return (p @ v) / l, (2 * rel + part) * weighted


def put(c, cache, tokens, row):
    """`row` in the cache, for `tokens` of the first sequence."""
    S = c.k.shape[1]
    at = torch.tensor([[c.table[0][j // S], j % S] for j in tokens], device="cuda").t()
    as_bytes = (lambda x: x.view(torch.uint8)) if cache.dtype == E4M3 else (lambda x: x)
    as_bytes(cache)[at[0], at[1]] = as_bytes(row.cuda().to(cache.dtype))


def rounded(y, err):
    """The bound with the rounding to bf16: half a step of the value's own binade,
    2^-8 to 2^-9 of it."""
    return err + torch.exp2(torch.floor(torch.log2((y.abs() + err).clamp(min=2.0 ** -120))) - 8)


# rows that share a key head, with two parts of 16 bits per weight: bf16 each
# leaves 2^-8 of what it rounds
TWO = 2.0 ** -16


@pytest.mark.parametrize("ct", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [6, 16])
def test_weights_of_up_to_16_rows_are_not_rounded_to_16_bits(ct, D, rows):
    """Small scores: weights between a half and one, that differ."""
    g = generator(D + rows)
    lens = [40, 150]
    c = Cache(g, lens, 16, 1, D, ct)
    q = normal(g, 2, rows, D, std=0.1)
    out, _ = attend(q, c, lens)
    for n, length in enumerate(lens):
        y, e = exact(q[n], c, n, length, D ** -0.5, TWO)
        check(out[n], y, rounded(y, e))


@pytest.mark.parametrize("ct", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [8, 16])
def test_one_token_that_outweighs_the_rest(ct, D, rows):
    """Weights of one, and one in a later tile of 2^4 to 2^7.5: little enough
    that the running maximum may lag behind it, so that its weight is no power
    of two.  Sequences enough (of the same tokens) that warps have whole ones."""
    g, N = generator(D + rows), 1600
    c = Cache(g, [200], 16, 1, D, ct)
    c.page_table = c.page_table.expand(N, -1).contiguous()
    for name in c.scales:
        c.scales[name] = torch.ones(1, device="cuda")
    put(c, c.k, range(200), torch.zeros(D))
    put(c, c.v, range(200), torch.full((D,), 2.0 ** -8))
    one = torch.zeros(D)
    one[0] = 1.0
    put(c, c.k, [149], one)
    put(c, c.v, [149], normal(g, D, dtype=F32))
    q = torch.zeros(N, rows, D, dtype=BF16, device="cuda")
    q[..., 0] = torch.linspace(4.0, 7.5, rows)
    out, _ = attend(q, c, [200] * N, scale=math.log(2.0))
    y, e = exact(q[0], c, 0, 200, math.log(2.0), TWO)
    check(out, y.expand(N, -1, -1), rounded(y, e))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [8, 16, 24, 64])
@pytest.mark.parametrize("nats", [12.0, 14.0, 16.0])
def test_many_small_weights_beside_a_large_one_over_8_bits(D, rows, nats):
    """A leading token of value zero that outweighs each of the others by e^12
    to e^16: the result is what the small ones bring.  Sequences enough (of the
    same tokens) that warps have whole ones."""
    N, length = 1600, 300
    c = Cache(generator(D), [length], 16, 1, D, E4M3)
    c.page_table = c.page_table.expand(N, -1).contiguous()
    for name in c.scales:
        c.scales[name] = torch.ones(1, device="cuda")
    put(c, c.k, range(length), torch.zeros(D))
    put(c, c.v, range(length), 1.0 + torch.arange(D) % 8 / 8)
    one = torch.zeros(D)
    one[0] = 1.0
    put(c, c.k, [0], one)
    put(c, c.v, [0], torch.zeros(D))
    q = torch.zeros(N, rows, D, dtype=BF16, device="cuda")
    q[..., 0] = nats
    out, lse = attend(q, c, [length] * N, scale=1.0)
    # Two parts of fp16 or one, and 2^-25 at the weights' scale of 2^7 for each.
    y, e = exact(q[0], c, 0, length, 1.0, 2.0 ** -22 if rows <= 16 else 2.0 ** -11)
    v = c.v.view(torch.uint8)[c.table[0][0], 1, 0].view(E4M3).double()
    e = e + 2.0 ** -32 * (length - 1) * v
    check(out, y.expand(N, -1, -1), rounded(y, e))
    want = math.log(1.0 + (length - 1) * math.exp(-nats)) + nats
    assert float((lse.double() - want).abs().max()) <= (12 + 3 * length) * U * want


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L,rows", [(1, 3), (1, 8), (1, 16), (1, 24), (4, 1), (4, 4), (8, 8)])
@pytest.mark.parametrize("length", [1, 40, 300])
def test_infinite_values_are_infinite_for_the_rows_that_see_them(dtype, D, L, rows, length):
    """A value of infinity, with weights of one and others: of the first, the
    newest or any token between."""
    g = generator(D + rows)
    N = 4
    c = Cache(g, [length] * N, 16, 1, D, dtype)
    q = normal(g, N, L, rows, D, dtype=dtype, std=0.3)
    q[1] = 0.0  # weights of one
    for n, j in enumerate((0, length // 2, length - 1, length - 1)):
        c.v[c.table[n][j // 16], j % 16, 0, 5] = math.inf
        c.v[c.table[n][j // 16], j % 16, 0, 8] = -math.inf
    out, lse = attend(q, c, [length] * N)
    for n, j in enumerate((0, length // 2, length - 1, length - 1)):
        for t in range(L):
            sees = length - L + t
            if sees < 0:
                assert (out[n, t] == 0).all()
                continue
            assert torch.isfinite(lse[n, t]).all()
            if sees >= j:
                assert (out[n, t, :, 5] == math.inf).all() and (out[n, t, :, 8] == -math.inf).all()
                out[n, t, :, [5, 8]] = 0.0
            assert torch.isfinite(out[n, t]).all()


@pytest.mark.parametrize("ct", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [8, 24])
@pytest.mark.parametrize("power", [24, 25, 26, 30])
def test_scores_too_large_for_steps_of_one(ct, rows, power):
    """Scores of 2^power and some more, in powers of two, where a step of fp32 is
    one or far more: whatever the weights come to, the result lies between the
    values.  Sequences enough that warps have whole ones."""
    N, length = 1600, 300
    c = Cache(generator(power), [length], 16, 1, 64, ct)
    c.page_table = c.page_table.expand(N, -1).contiguous()
    for name in c.scales:
        c.scales[name] = torch.ones(1, device="cuda")
    put(c, c.v, range(length), 1.0 + torch.arange(64) % 8 / 8)
    key = torch.zeros(64)
    key[0] = 256.0
    q = torch.zeros(N, rows, 64, dtype=BF16, device="cuda")
    q[..., 0] = 2.0 ** (power - 8)
    q[..., 1] = 2.0 ** (power - 24)
    for step in range(0, 64, 4):  # the later tiles' scores: that of the first and up to 2^(power - 18) more
        put(c, c.k, range(length), key)
        later = key.clone()
        later[1] = step
        put(c, c.k, range(70, length), later)
        out, lse = attend(q, c, [length] * N, scale=math.log(2.0))
        assert torch.isfinite(lse).all()
        want = (1.0 + torch.arange(64, device="cuda") % 8 / 8).double()
        assert float(((out.double() - want).abs() / want).max()) <= 2.0 ** -6, step
