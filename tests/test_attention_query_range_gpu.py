"""Queries of any magnitude beside an 8-bit cache, whose products take them as fp16
over a power of two of their row's largest."""
import math

import pytest
import torch

from test_attention_ops_gpu import BF16, E4M3, Cache, attend, check_attention, generator, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("power", [-126, -121, -60, 0, 60, 119, 120, 121, 125])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("D,rows", [(64, 5), (128, 16), (256, 48)])
def test_queries_of_any_magnitude(power, sign, D, rows):
    """Queries of about 2^power, keys scaled the other way: scores of the usual
    size."""
    g = generator(D)
    lens = [100, 33]
    c = Cache(g, lens, 16, 1, D, E4M3)
    by = min(max(power, -100), 100)  # the keys' part of it; the scale has the rest
    c.scales["k_scale"] = c.scales["k_scale"] * 2.0 ** -by
    q = (normal(g, 2, rows, D, dtype=torch.float32).clamp(-3, 3) * 2.0 ** power).to(BF16)
    scale = sign * D ** -0.5 * 2.0 ** (by - power)
    check_attention(q, c, lens, attend(q, c, lens, scale=scale), scale=scale)


@pytest.mark.parametrize("power", [0, 119, 126])
def test_an_infinite_query_spoils_its_row_alone(power):
    """Keys of one sign, so that the row's scores are all infinite: NaN, or of
    -infinity alone: nothing.  Rows beside it, large ones too, do not show it."""
    g = generator(power)
    lens = [70]
    c = Cache(g, lens, 16, 1, 64, E4M3)
    c.k.view(torch.uint8).copy_(c.k.float().abs().clamp(1, 400).to(E4M3).view(torch.uint8))
    c.scales["k_scale"] = torch.full((1,), 2.0 ** -power, device="cuda")
    q = (normal(g, 1, 4, 64, dtype=torch.float32).clamp(-3, 3) * 2.0 ** power).to(BF16)
    want = attend(q, c, lens, scale=0.1)
    for value in (math.inf, -math.inf, math.nan):
        x = q.clone()
        x[0, 2, 9] = value
        out, lse = attend(x, c, lens, scale=0.1)
        if value == -math.inf:
            assert (out[0, 2] == 0).all() and lse[0, 2] == -math.inf
        else:
            assert torch.isnan(out[0, 2]).all() and torch.isnan(lse[0, 2])
        for got, w in zip((out, lse), want):
            assert torch.equal(got[0, [0, 1, 3]], w[0, [0, 1, 3]])
