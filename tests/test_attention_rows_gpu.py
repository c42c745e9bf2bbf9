"""A row's result and statistics are its own: bit for bit the same whatever the
rows beside it see."""
import pytest
import torch

from test_attention_ops_gpu import BF16, E4M3, F32, Cache, attend, bits, generator, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dtype,ct", [(BF16, BF16), (BF16, E4M3), (F32, F32)], ids=["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L,G", [(2, 2), (4, 2), (4, 4), (4, 6), (8, 4), (8, 6), (8, 12)])
def test_large_scores_of_later_tokens_do_not_show(dtype, ct, D, L, G):
    """The newest token's key, which the last row alone sees, is made large: the
    rows before it keep every bit of their results and log-sum-exps."""
    g = generator(D + L * G)
    N, lens = 40, [300] * 40
    c = Cache(g, lens, 16, 1, D, ct)
    q = normal(g, N, L, G, D, dtype=dtype)
    want = attend(q, c, lens)
    for n in range(N):
        at = c.k[c.table[n][299 // 16]]
        row = (q[n, L - 1, 0].float() * (4.0 if ct == E4M3 else 2.0)).clamp(-448, 448).to(ct)
        if ct == E4M3:
            at.view(torch.uint8)[299 % 16, 0] = row.view(torch.uint8)
        else:
            at[299 % 16, 0] = row
    got = attend(q, c, lens)
    assert not torch.equal(got[1][:, L - 1], want[1][:, L - 1])
    for a, b in zip(got, want):
        assert torch.equal(bits(a[:, :L - 1]), bits(b[:, :L - 1]))
