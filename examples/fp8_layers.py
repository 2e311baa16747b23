"""A feed-forward block's training step and an expert block's decoding step on 8-bit matrices.

    python examples/fp8_layers.py [--tokens 4096] [--hidden 2048] [--inner 4096] [--experts 16] [--steps 20]

Training: RMS norm with residual addition and 8-bit output, a linear layer whose three products (output, input
gradient, weight gradient) run on 8-bit codes, and the norm's gradient; the weights are kept in FP32 and quantised once
per step.  Decoding: the same norm, a router's logits and the experts' layer, captured in one CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sgemm_row_major_gb300 as sg  # noqa: E402


class NormLinear:
    """out = rmsnorm(x + residual) W^T, on 8-bit codes of the norm's output and of W."""

    def __init__(self, inputs: int, outputs: int, generator):
        self.weight = torch.randn(outputs, inputs, device="cuda", generator=generator) * inputs ** -0.5
        self.gain = torch.ones(inputs, device="cuda", dtype=torch.bfloat16)
        self.quantise()

    def quantise(self):
        self.codes = sg.quantize_fp8(self.weight, (128, 128))

    def forward(self, x, residual):
        n = sg.rmsnorm_fp8(x, self.gain, 1e-6, residual, y=True)
        self.saved = n
        return sg.matmul_fp8(n.q, self.codes, transB="T", out_dtype=torch.bfloat16), n.h

    def backward(self, dout, dh):
        """(gradient of x and of the residual, of the weight, of the gain); dh: the gradient of the returned sum."""
        n = self.saved
        dy = sg.matmul_fp8(sg.quantize_fp8(dout, format="e5m2"), self.codes, out_dtype=torch.bfloat16)
        dweight = sg.matmul_fp8(sg.quantize_fp8(dout, (128, 1), "e5m2"), sg.quantize_fp8(n.y, (128, 1)), transA="T")
        dx, dgain = sg.rmsnorm_fp8_backward(dy, n.h, self.gain, n.rstd, dh)
        return dx, dweight, dgain


def train(tokens=4096, hidden=2048, outputs=4096, steps=20, rate=0.25, seed=0):
    """Losses of `steps` steps of plain gradient descent towards another layer's outputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    layer, target = NormLinear(hidden, outputs, g), NormLinear(hidden, outputs, g)
    x, residual = (torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16() for _ in range(2))
    want, _ = target.forward(x, residual)
    losses = []
    for _ in range(steps):
        out, h = layer.forward(x, residual)
        diff = out.float() - want.float()
        losses.append(diff.square().mean())
        dout = (diff * (2.0 / tokens)).bfloat16()  # of the mean over tokens of the summed squares
        _, dweight, dgain = layer.backward(dout, torch.zeros_like(h))
        layer.weight -= rate * dweight
        layer.gain -= (rate / outputs * dgain).bfloat16()
        layer.quantise()
    return [float(v) for v in losses]


class ExpertBlock:
    """x + residual, its RMS norm, and the top_k experts of each token: what a decoding step does after attention."""

    def __init__(self, hidden: int, inner: int, experts: int, top_k: int, generator):
        def stack(rows, cols):
            made = [sg.quantize_fp8(torch.randn(rows, cols, device="cuda", generator=generator) * cols ** -0.5, (128, 128))
                    for _ in range(experts)]
            return torch.stack([m.data for m in made]), torch.stack([m.scale for m in made])

        self.gain = torch.ones(hidden, device="cuda", dtype=torch.bfloat16)
        self.router = torch.randn(experts, hidden, device="cuda", generator=generator) * hidden ** -0.5
        self.gate, self.up, self.down = stack(inner, hidden), stack(inner, hidden), stack(hidden, inner)
        self.top_k = top_k

    def __call__(self, x, residual):
        n = sg.rmsnorm_fp8(x, self.gain, 1e-6, residual, y=True)
        logits = torch.empty(x.shape[0], self.router.shape[0], device="cuda")
        sg.matmul(n.y.float(), self.router, logits, "N", "T", 1.0, 0.0)
        return sg.moe_fp8(n.q, logits, self.top_k, self.gate, self.up, self.down), n.h


def decode(tokens=8, hidden=2048, inner=4096, experts=16, top_k=2, steps=20, seed=0):
    """The hidden states after `steps` applications of one expert block, by graph replay, and the time of one (us)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    block = ExpertBlock(hidden, inner, experts, top_k, g)
    x = torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16()
    state = torch.zeros_like(x)
    block(x, state)  # first calls load the kernels
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, h = block(x, state)
        state.copy_(h)
        x.copy_(out)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return x, state, begin.elapsed_time(end) * 1e3 / max(steps, 1)


def main() -> None:
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--tokens", type=int, default=4096)
    a.add_argument("--hidden", type=int, default=2048)
    a.add_argument("--inner", type=int, default=4096)
    a.add_argument("--experts", type=int, default=16)
    a.add_argument("--steps", type=int, default=20)
    a = a.parse_args()
    losses = train(a.tokens, a.hidden, a.inner, a.steps)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    x, state, us = decode(hidden=a.hidden, inner=a.inner, experts=a.experts, steps=a.steps)
    print(f"decoding: 8 tokens, {us:.1f} us a step, |h| {float(state.float().norm()):.3f}")


if __name__ == "__main__":
    main()
