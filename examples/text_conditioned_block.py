#!/usr/bin/env python3
"""A text-conditioned diffusion-transformer block on libternary: ternary linear
layers with the operators that stand between them.

One block, for image tokens x on a frames x height x width grid and padded
caption states:

  x, h = boundary(x)                  norm, modulated by the conditioning
  q, k, v = ternary(h)                rotary positions (time, height, width) on q, k
  x, h = boundary(x, ternary(attention(q, k, v)))      gate, residual, next norm
  x, h = boundary(x, ternary(attention(ternary(h), caption)))
  x    = boundary(x, ternary(gelu(ternary(h))))

Every weight of a linear layer is a latent full-precision matrix that is
ternarized in the forward pass and trained straight through.  Run as a program
it trains one block on a synthetic target for a few steps:

  python examples/text_conditioned_block.py [--steps 20] [--hidden 1152] [--heads 16]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ternary_weight_quantized_tern_amd as tern  # noqa: E402


def rotary_axes(width: int):
    """Channels of a head for time, height and width: a quarter and two equal
    parts, all even."""
    side = (width * 3 // 8) // 2 * 2
    return (width - 2 * side, side, side)


def grid_positions(frames: int, height: int, width: int, device) -> torch.Tensor:
    axes = [torch.arange(n, device=device, dtype=torch.float32) for n in (frames, height, width)]
    return torch.stack(torch.meshgrid(*axes, indexing="ij"), dim=-1).reshape(-1, 3)


class Block(torch.nn.Module):
    """hidden and the MLP width are multiples of 64 (the ternary layer's rule)."""

    def __init__(self, hidden: int, heads: int, conditioning: int):
        super().__init__()
        self.heads, self.width = heads, hidden // heads
        self.axes = rotary_axes(self.width)

        def weight(n, k):
            return torch.nn.Parameter(0.02 * torch.randn(n, k))

        self.qkv = weight(3 * hidden, hidden)
        self.out = weight(hidden, hidden)
        self.cross_q = weight(hidden, hidden)
        self.cross_kv = weight(2 * hidden, hidden)
        self.cross_out = weight(hidden, hidden)
        self.up = weight(4 * hidden, hidden)
        self.down = weight(hidden, 4 * hidden)
        # scale, shift and gate of the three sub-blocks
        self.modulation = torch.nn.Linear(conditioning, 9 * hidden)

    def forward(self, x, caption, caption_mask, positions, conditioning):
        """x [b, t, hidden] (fp32 or bf16), caption [b, s, hidden] bf16,
        caption_mask [b, s], positions [t, 3], conditioning [b, c]."""
        b, t, c = x.shape
        s = caption.shape[1]
        mod = self.modulation(conditioning).split(c, dim=1)
        (scale1, shift1, gate1), (scale2, shift2, gate2), (scale3, shift3, gate3) = (
            mod[0:3], mod[3:6], mod[6:9])
        r = x.reshape(b * t, c)

        h = tern.block_boundary(r, scale=scale1, shift=shift1, tokens=t)
        qkv = tern.ternary_linear(h, self.qkv).view(b, t, 3 * self.heads, self.width)
        qk, v = qkv[:, :, :2 * self.heads], qkv[:, :, 2 * self.heads:]
        qk = tern.rotary(qk, positions, self.axes)
        o = tern.cross_attention(qk[:, :, :self.heads], qk[:, :, self.heads:], v)
        y = tern.ternary_linear(o.reshape(b * t, c), self.out)

        r, h = tern.block_boundary(r, y, gate=gate1, scale=scale2, shift=shift2, tokens=t)
        q = tern.ternary_linear(h, self.cross_q).view(b, t, self.heads, self.width)
        kv = tern.ternary_linear(caption.reshape(b * s, c), self.cross_kv)
        kv = kv.view(b, s, 2 * self.heads, self.width)
        o = tern.cross_attention(q, kv[:, :, :self.heads], kv[:, :, self.heads:],
                                 mask=caption_mask)
        y = tern.ternary_linear(o.reshape(b * t, c), self.cross_out)

        r, h = tern.block_boundary(r, y, gate=gate2, scale=scale3, shift=shift3, tokens=t)
        y = torch.nn.functional.gelu(tern.ternary_linear(h, self.up), approximate="tanh")
        y = tern.ternary_linear(y, self.down)
        return tern.block_boundary(r, y, gate=gate3, tokens=t, pre=None).view(b, t, c)


def train(steps: int = 20, hidden: int = 1152, heads: int = 16, batch: int = 4, grid=(1, 16, 16),
          states: int = 120, seed: int = 0):
    """A few steps of the block towards a fixed random target; returns the losses."""
    dev = "cuda"
    torch.manual_seed(seed)
    tokens = grid[0] * grid[1] * grid[2]
    block = Block(hidden, heads, 256).to(dev)
    optimizer = torch.optim.Adam(block.parameters(), lr=1e-3)
    x = torch.randn(batch, tokens, hidden, device=dev)
    caption = torch.randn(batch, states, hidden, device=dev).to(torch.bfloat16)
    length = torch.randint(1, states + 1, (batch, 1), device=dev)
    length[-1] = 0  # a dropped caption: nothing to attend to
    mask = torch.arange(states, device=dev)[None] < length
    conditioning = torch.randn(batch, 256, device=dev)
    positions = grid_positions(*grid, dev)
    target = torch.randn(batch, tokens, hidden, device=dev)
    losses = []
    for _ in range(steps):
        loss = (block(x, caption, mask, positions, conditioning) - target).square().mean()
        optimizer.zero_grad(set_to_none=True)
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
    return [float(v) for v in losses]


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--hidden", type=int, default=1152)
    p.add_argument("--heads", type=int, default=16)
    p.add_argument("--batch", type=int, default=4)
    a = p.parse_args()
    losses = train(a.steps, a.hidden, a.heads, a.batch)
    print("loss " + " ".join("%.4f" % v for v in losses))


if __name__ == "__main__":
    main()
