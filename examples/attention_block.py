"""A gated attention block served with the library's operators.

The block is the one that hybrid models put between their fixed-state layers:
norm, projection to queries with their output gates, keys and values, norms and
rotation of queries and keys for each head, attention over a paged cache, output
projection, then the norm and residual that lead to the next block.  The
projections are plain matrix products, a prompt's attention over itself is
PyTorch's; everything else is

    gdn_qk_norm_rope    gdn_paged_append    gdn_paged_attention
    gdn_norm_gate_residual

``prompt`` takes packed prompts of any lengths, ``tokens`` one to eight new
tokens of each sequence.  Run as a program, it serves a batch of ragged prompts
and a few tokens and compares them with the same sequences taken as longer
prompts:

    python examples/attention_block.py [--model 512] [--steps 6] [--drafted 2]
"""
from __future__ import annotations

import argparse
import os
import sys
from typing import List, Tuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_chunk_gb300 as gdn  # noqa: E402


class Cache:
    """Pages for `sequences` of up to `room` tokens; a page holds its tokens
    head by head."""

    def __init__(self, block: "AttentionBlock", sequences: int, room: int, page_size: int = 16):
        each = -(-room // page_size)
        shape = (sequences * each, block.kv_heads, page_size, block.head_dim)
        self.k, self.v = (torch.empty(shape, dtype=block.dtype, device="cuda").transpose(1, 2)
                          for _ in range(2))
        order = torch.randperm(sequences * each).to(torch.int32)
        self.page_table = order.view(sequences, each).cuda()
        self.seq_lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")

    def args(self):
        return dict(k_cache=self.k, v_cache=self.v, page_table=self.page_table,
                    seq_lens=self.seq_lens)


class AttentionBlock:
    """Random weights of one block."""

    def __init__(self, model: int, heads: int = 6, kv_heads: int = 1, head_dim: int = 128,
                 rotary: int = 32, dtype=torch.bfloat16, seed: int = 0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(*shape, std, dtype=dtype):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)
        f32 = torch.float32
        self.heads, self.kv_heads, self.head_dim, self.dtype = heads, kv_heads, head_dim, dtype
        self.w_in = normal(model, 2 * (heads + kv_heads) * head_dim, std=model ** -0.5)
        self.w_out = normal(heads * head_dim, model, std=(heads * head_dim) ** -0.5)
        self.q_weight, self.k_weight = (1.0 + normal(head_dim, std=0.1, dtype=f32) for _ in range(2))
        self.inv_freq = 1e6 ** (-torch.arange(0, rotary, 2, device="cuda", dtype=f32) / rotary)
        self.next_norm_w = torch.ones(model, device="cuda")

    def _project(self, h: torch.Tensor):
        """Queries beside their gates head by head, keys and values: all are
        views of one projection."""
        x = h @ self.w_in
        qg, k, v = x.split([2 * self.heads * self.head_dim] + 2 * [self.kv_heads * self.head_dim], 1)
        qg = qg.unflatten(1, (self.heads, 2 * self.head_dim))
        k, v = (t.unflatten(1, (self.kv_heads, self.head_dim)) for t in (k, v))
        return qg[..., :self.head_dim], qg[..., self.head_dim:], k, v

    def _leave(self, y: torch.Tensor, residual: torch.Tensor):
        return gdn.gdn_norm_gate_residual(y.flatten(1) @ self.w_out, residual=residual,
                                          next_weight=self.next_norm_w)

    def prompt(self, h: torch.Tensor, residual: torch.Tensor, lens: List[int], cache: Cache):
        """Packed prompts, from the sequences' first tokens on: h (normed) and
        residual [T, model].  Returns (residual, normed input of the next
        block)."""
        q, gate, k, v = self._project(h)
        cu = torch.tensor([0] + lens).cumsum(0)
        positions = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
        q, k = gdn.gdn_qk_norm_rope(q, k, positions, self.inv_freq, self.q_weight, self.k_weight)
        cache.seq_lens.copy_(torch.tensor(lens))
        gdn.gdn_paged_append(k, v, cu_seqlens=cu.to(torch.int32).cuda(), **cache.args())
        y = torch.empty_like(q)
        for b, e in zip(cu[:-1].tolist(), cu[1:].tolist()):
            if e > b:
                y[b:e] = torch.nn.functional.scaled_dot_product_attention(
                    *(t[b:e].transpose(0, 1)[None] for t in (q, k, v)), is_causal=True,
                    enable_gqa=True)[0].transpose(0, 1)
        return self._leave(y * torch.sigmoid(gate.float()).to(y.dtype), residual)

    def tokens(self, h: torch.Tensor, residual: torch.Tensor, cache: Cache):
        """New tokens of each sequence, L each: h and residual [N L, model]."""
        sequences = cache.seq_lens.shape[0]
        cache.seq_lens.add_(h.shape[0] // sequences)
        q, gate, k, v = self._project(h)
        q = gdn.gdn_paged_append(k, v, q=q, inv_freq=self.inv_freq, q_weight=self.q_weight,
                                 k_weight=self.k_weight, **cache.args())
        y = gdn.gdn_paged_attention(q.unflatten(0, (sequences, -1)), gate=gate.unflatten(0, (sequences, -1)),
                                    **cache.args())
        return self._leave(y.flatten(0, 1), residual)


def serve(block: AttentionBlock, lens: List[int], steps: int, drafted: int, model: int,
          seed: int = 1) -> Tuple[float, float]:
    """Serves prompts of `lens`, then `steps` times `drafted` tokens of each,
    and the whole sequences as prompts; returns (largest difference of the next
    block's inputs, their largest value)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    more = steps * drafted
    whole = [n + more for n in lens]
    ends = torch.tensor(whole).cumsum(0).tolist()
    starts = [e - n for e, n in zip(ends, whole)]
    residual = torch.randn(sum(whole), model, generator=gen, device="cuda").to(block.dtype)
    _, h = gdn.gdn_norm_gate_residual(residual, next_weight=block.next_norm_w)
    _, want = block.prompt(h, residual, whole, Cache(block, len(lens), max(whole)))

    cache, got = Cache(block, len(lens), max(whole)), torch.empty_like(want)
    rows = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, lens)]).cuda()
    _, got[rows] = block.prompt(h[rows], residual[rows], lens, cache)
    for t in range(0, more, drafted):
        rows = torch.cat([torch.arange(drafted) + s + n + t for s, n in zip(starts, lens)]).cuda()
        _, got[rows] = block.tokens(h[rows], residual[rows], cache)
    return float((got.float() - want.float()).abs().max()), float(want.float().abs().max())


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--model", type=int, default=512)
    ap.add_argument("--steps", type=int, default=6)
    ap.add_argument("--drafted", type=int, default=2)
    a = ap.parse_args()
    lens = [257, 1, 64, 1000, 5]
    off, most = serve(AttentionBlock(a.model), lens, a.steps, a.drafted, a.model)
    print(f"prompts of {lens} tokens and {a.steps} x {a.drafted} tokens each, against whole prompts:")
    print(f"  next block's input: largest difference {off:.3g} of values up to {most:.3g}")


if __name__ == "__main__":
    main()
