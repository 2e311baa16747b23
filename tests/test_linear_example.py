"""The example on BF16 layers: it runs, and its gradients are those of the block."""
import importlib.util
import os

import pytest

import sgemm_row_major_gb300 as sg

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("bf16_block", os.path.join(ROOT, "examples", "bf16_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_it_runs(example):
    import math
    losses = example.train(300, 256, 384, steps=2)
    assert len(losses) == 2 and all(math.isfinite(v) for v in losses)
    assert sg.sgemm_sync_status() == 0


def test_gradients(example):
    """Against autograd in 64 bits of the same block.  What the backward pass reads in 8 bits is off by 2^-4 of itself at most,
    each independently, so sums of hundreds of terms are off by a few hundredths of their norm; a missing or wrong term would
    be off by about all of it."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    block = example.GatedBlock(256, 384, g)
    x = torch.randn(300, 256, device="cuda", generator=g).bfloat16()
    dy = (torch.randn(300, 256, device="cuda", generator=g) * 0.1).bfloat16()
    y = block.forward(x)
    got = block.backward(dy)
    leaves = [v.double().requires_grad_() for v in (x, block.gain, block.gate, block.up, block.down)]
    x_, gain, gate, up, down = leaves
    n = x_ * (x_.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gain
    h = torch.nn.functional.silu(n @ gate.T) * (n @ up.T)
    out = x_ + h @ down.T
    # n, h and y are each rounded to BF16 once: 2^-8 of themselves, less in norm
    assert float((y.double() - out).norm() / out.norm()) <= 2.0 ** -8
    want = torch.autograd.grad(out, leaves, dy.double())
    for name, a, b in zip(("x", "gain", "gate", "up", "down"), got, want):
        assert a.shape == b.shape
        assert float((a.double() - b).norm() / b.norm()) <= 2.0 ** -4, name
    assert sg.sgemm_sync_status() == 0
