"""A selective state space block served with the library's operators.

The block is the other fixed-state layer of hybrid models, beside Gated
DeltaNet: norm, projection, short causal convolution, selective scan, output
projection, then the norm and residual that lead to the next block.  The
projections are plain matrix products; everything between them is

    gdn_short_conv          gdn_short_conv_step
    gdn_selective_scan      gdn_selective_scan_step
    gdn_norm_gate_residual

``prompt`` takes packed prompts of any lengths and leaves each sequence's
convolution window and state; ``token`` takes one token of each sequence from
there.  Run as a program, it serves a batch of ragged prompts and a few tokens
and compares them with the same sequences taken as longer prompts:

    python examples/selective_block.py [--model 512] [--channels 1024] [--tokens 8]
"""
from __future__ import annotations

import argparse
import os
import sys
from typing import List, Tuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_chunk_gb300 as gdn  # noqa: E402


class SelectiveBlock:
    """Random weights of one block: ``model`` is the residual stream's width,
    ``channels`` the scan's, with ``states`` per channel."""

    def __init__(self, model: int, channels: int, states: int = 16, width: int = 4,
                 dtype=torch.bfloat16, device="cuda", seed: int = 0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def normal(*shape, std, dtype=dtype):
            return (torch.randn(*shape, generator=gen, device=device) * std).to(dtype)
        f32 = torch.float32
        self.channels, self.states, self.width, self.dtype = channels, states, width, dtype
        self.w_in = normal(model, 2 * channels, std=model ** -0.5)
        self.conv_w = normal(channels, width, std=width ** -0.5, dtype=f32)
        self.conv_b = normal(channels, std=0.1, dtype=f32)
        self.rank = max(8, channels // 16)
        self.w_x = normal(channels, self.rank + 2 * states, std=channels ** -0.5)
        self.w_dt = normal(self.rank, channels, std=0.5 * self.rank ** -0.5)
        # Steps log-uniform over [0.001, 0.1], decay rates 1 .. states.
        step = torch.exp(torch.empty(channels, device=device).uniform_(-6.9, -2.3, generator=gen))
        self.dt_bias = step + torch.log(-torch.expm1(-step))
        self.A = -torch.arange(1, states + 1, device=device, dtype=f32).repeat(channels, 1)
        self.D = torch.ones(channels, device=device)
        self.w_out = normal(channels, model, std=channels ** -0.5)
        self.norm_w = torch.ones(model, device=device)       # after the block
        self.next_norm_w = torch.ones(model, device=device)  # before the next

    def new_state(self, sequences: int) -> Tuple[torch.Tensor, torch.Tensor]:
        """Empty convolution windows and states."""
        dev = self.w_in.device
        return (torch.zeros(sequences, self.width - 1, self.channels, dtype=self.dtype, device=dev),
                torch.zeros(sequences, self.channels, self.states, device=dev))

    def _inputs(self, h: torch.Tensor):
        xz = h @ self.w_in
        return xz[:, :self.channels], xz[:, self.channels:]  # rows stay strided

    def _steps(self, x: torch.Tensor):
        low = x @ self.w_x
        B = low[:, self.rank:self.rank + self.states].unflatten(1, (1, self.states))
        C = low[:, self.rank + self.states:].unflatten(1, (1, self.states))
        return low[:, :self.rank] @ self.w_dt, B, C

    def _leave(self, y: torch.Tensor, residual: torch.Tensor):
        return gdn.gdn_norm_gate_residual(y @ self.w_out, self.norm_w, residual=residual,
                                          next_weight=self.next_norm_w)

    def prompt(self, h: torch.Tensor, residual: torch.Tensor, cu_seqlens: torch.Tensor, state):
        """Packed prompts: h (normed) and residual [T, model].  Updates the
        state in place; returns (residual, normed input of the next block)."""
        window, ssm = state
        x, z = self._inputs(h)
        x, _ = gdn.gdn_short_conv(x, self.conv_w, cu_seqlens, bias=self.conv_b,
                                  initial_state=window, final_state=window, activation="silu")
        dt, B, C = self._steps(x)
        y, _ = gdn.gdn_selective_scan(x, dt, self.A, B, C, cu_seqlens, D=self.D, z=z,
                                      dt_bias=self.dt_bias, dt_softplus=True, initial_state=ssm,
                                      final_state=ssm)
        return self._leave(y, residual)

    def token(self, h: torch.Tensor, residual: torch.Tensor, state):
        """One token of each sequence: h and residual [N, model]."""
        window, ssm = state
        x, z = self._inputs(h)
        x = gdn.gdn_short_conv_step(x, self.conv_w, window, bias=self.conv_b, activation="silu")
        dt, B, C = self._steps(x)
        y = gdn.gdn_selective_scan_step(x, dt, self.A, B, C, ssm, D=self.D, z=z,
                                        dt_bias=self.dt_bias, dt_softplus=True)
        return self._leave(y, residual)


def cumulative(lens: List[int], device="cuda") -> torch.Tensor:
    return torch.tensor([0] + lens, device=device).cumsum(0).to(torch.int32)


def serve(block: SelectiveBlock, lens: List[int], tokens: int, model: int, seed: int = 1):
    """Serves prompts of `lens` and `tokens` further tokens of each, then the
    whole sequences as prompts; returns (largest difference of the next
    block's inputs, their largest value, the same of the states)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    whole = [n + tokens for n in lens]
    ends = torch.tensor(whole).cumsum(0).tolist()
    starts = [e - n for e, n in zip(ends, whole)]
    residual = torch.randn(sum(whole), model, generator=gen, device="cuda").to(block.dtype)
    _, h = gdn.gdn_norm_gate_residual(residual, next_weight=block.next_norm_w)

    state = block.new_state(len(lens))
    _, want = block.prompt(h, residual, cumulative(whole), state)

    rows = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, lens)]).cuda()
    served = block.new_state(len(lens))
    got = torch.empty_like(want)
    _, got[rows] = block.prompt(h[rows], residual[rows], cumulative(lens), served)
    for t in range(tokens):
        rows = torch.tensor([s + n + t for s, n in zip(starts, lens)]).cuda()
        _, got[rows] = block.token(h[rows], residual[rows], served)

    def off(a, b):
        return float((a.float() - b.float()).abs().max()), float(b.float().abs().max())
    return off(got, want), off(served[1], state[1])


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--model", type=int, default=512)
    ap.add_argument("--channels", type=int, default=1024)
    ap.add_argument("--tokens", type=int, default=8)
    a = ap.parse_args()
    block = SelectiveBlock(a.model, a.channels)
    lens = [257, 1, 64, 1000, 5]
    out, state = serve(block, lens, a.tokens, a.model)
    print(f"prompts of {lens} tokens and {a.tokens} tokens each, against whole prompts:")
    print(f"  next block's input: largest difference {out[0]:.3g} of values up to {out[1]:.3g}")
    print(f"  states:             largest difference {state[0]:.3g} of values up to {state[1]:.3g}")


if __name__ == "__main__":
    main()
