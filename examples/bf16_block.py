"""A gated feed-forward block's training step on BF16 weights, with what its backward pass needs kept in 8 bits.

    python examples/bf16_block.py [--tokens 4096] [--hidden 2048] [--inner 4096] [--steps 20]

Forward: RMS norm (whose output is kept as 8-bit codes alone), the gated half of the block in one kernel, which keeps both of
its products in 8 bits, and the layer behind it with the block's input added.  Backward: that layer's gradients, the gated
half's from the kept values (with its output made again for the weight gradient of the layer behind), and the norm's.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sgemm_row_major_gb300 as sg  # noqa: E402


class GatedBlock:
    """x + down(silu(gate n) * (up n)), n = rmsnorm(x)."""

    def __init__(self, hidden: int, inner: int, generator):
        def weight(rows, cols):
            return (torch.randn(rows, cols, device="cuda", generator=generator) * cols ** -0.5).bfloat16()

        self.gain = torch.ones(hidden, device="cuda", dtype=torch.bfloat16)
        self.gate, self.up, self.down = weight(inner, hidden), weight(inner, hidden), weight(hidden, inner)

    def forward(self, x):
        n = sg.rmsnorm_fp8(x, self.gain, y=True)
        mid = sg.gated_bf16(n.y, self.gate, self.up, save="fp8")
        # what stays of all between the block's input and output: a byte per hidden value and two per inner one, and their scales
        self.saved = x, n.q, n.rstd, mid.gate, mid.up
        return sg.linear_bf16(mid.h, self.down, residual=x).y

    def backward(self, dy):
        """(gradient of x, of the gain, of gate, of up, of down)."""
        x, q, rstd, a, b = self.saved
        dh = sg.linear_bf16_backward(dy, None, self.down, dweight=False).dx
        g = sg.gated_bf16_backward(dh, q, self.gate, self.up, a, b, h=True)
        ddown = sg.linear_bf16_backward(dy, g.h, None, dx=False).dweight
        dx, dgain = sg.rmsnorm_fp8_backward(g.dx, x, self.gain, rstd, dy)
        return dx, dgain, g.dgate, g.dup, ddown


def train(tokens=4096, hidden=2048, inner=4096, steps=20, rate=0.5, seed=0):
    """Losses of `steps` steps of plain gradient descent towards another block's outputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    block, target = GatedBlock(hidden, inner, g), GatedBlock(hidden, inner, g)
    x = torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16()
    want = target.forward(x)
    losses = []
    for _ in range(steps):
        diff = block.forward(x).float() - want.float()
        losses.append(diff.square().mean())
        _, dgain, dgate, dup, ddown = block.backward((diff * (2.0 / tokens)).bfloat16())  # mean over tokens of the summed squares
        block.gain -= (rate / hidden * dgain).bfloat16()
        for w, d in ((block.gate, dgate), (block.up, dup), (block.down, ddown)):
            w -= rate * d
    return [float(v) for v in losses]


def main() -> None:
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--tokens", type=int, default=4096)
    a.add_argument("--hidden", type=int, default=2048)
    a.add_argument("--inner", type=int, default=4096)
    a.add_argument("--steps", type=int, default=20)
    a = a.parse_args()
    losses = train(a.tokens, a.hidden, a.inner, a.steps)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")


if __name__ == "__main__":
    main()
