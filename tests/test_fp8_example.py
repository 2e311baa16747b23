"""The 8-bit operators together, as examples/fp8_layers.py uses them, against the same steps in 64 bits."""
import os
import sys

import pytest

import sgemm_row_major_gb300 as sg
from fp8_util import dequantize

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


BF16 = 2.0 ** -8  # unit roundoff: 8 significant bits


def real(m):
    """The values of an Fp8Matrix in 64 bits."""
    import torch
    return torch.from_numpy(dequantize(m))


def close(got, want, mag, rel):
    """|got - want| <= rel * mag element by element."""
    err = (got.double().cpu() - want).abs()
    assert bool((err <= rel * mag).all()), float((err / mag).max())


@pytest.mark.gpu
def test_training_step():
    """Each product and gradient of one step against the formula on the codes that went in: FP32 sums ((K + 2) 2^-24
    of the absolute sum) and one rounding to BF16."""
    import torch
    import fp8_layers
    g = torch.Generator(device="cuda").manual_seed(1)
    T, I, O = 200, 384, 272
    layer = fp8_layers.NormLinear(I, O, g)
    x, r = (torch.randn(T, I, device="cuda", generator=g).bfloat16() for _ in range(2))
    dout, dh = torch.randn(T, O, device="cuda", generator=g).bfloat16(), torch.randn(T, I, device="cuda", generator=g).bfloat16()
    out, h = layer.forward(x, r)
    dx, dweight, dgain = layer.backward(dout, dh)
    n = layer.saved
    q, w = real(n.q), real(layer.codes)
    close(out, q @ w.T, q.abs() @ w.abs().T, BF16 + (I + 2) * 2.0 ** -24)
    hd = x.double().cpu() + r.double().cpu()
    close(h, hd, hd.abs(), BF16 + 2.0 ** -24)
    d8, dc, yc = real(sg.quantize_fp8(dout, format="e5m2")), real(sg.quantize_fp8(dout, (128, 1), "e5m2")), real(sg.quantize_fp8(n.y, (128, 1)))
    close(dweight, dc.T @ yc, dc.abs().T @ yc.abs(), (T + 2) * 2.0 ** -24)
    dy = sg.matmul_fp8(sg.quantize_fp8(dout, format="e5m2"), layer.codes, out_dtype=torch.bfloat16).double().cpu()
    close(dy, d8 @ w, d8.abs() @ w.abs(), BF16 + (O + 2) * 2.0 ** -24)
    hb, gain, rstd = h.double().cpu(), layer.gain.double().cpu(), n.rstd.double().cpu()[:, None]
    gw = dy * gain
    want = rstd * (gw - hb * rstd ** 2 * (gw * hb).mean(1, keepdim=True)) + dh.double().cpu()
    mag = rstd * (gw.abs() + hb.abs() * rstd ** 2 * (gw * hb).abs().mean(1, keepdim=True)) + dh.double().cpu().abs()
    close(dx, want, mag, BF16 + (I + 16) * 2.0 ** -24)
    close(dgain, (dy * hb * rstd).sum(0), (dy * hb * rstd).abs().sum(0), (T + 8) * 2.0 ** -24)


@pytest.mark.gpu
def test_training_learns():
    """Gradient descent on a layer's weights brings its outputs towards another's."""
    import fp8_layers
    losses = fp8_layers.train(tokens=512, hidden=256, outputs=384, steps=20)
    assert losses[-1] < 0.25 * losses[0] and all(b < a for a, b in zip(losses, losses[1:5])), losses


@pytest.mark.gpu
def test_decoding():
    """Replayed decoding steps are the same as eager ones, bit for bit."""
    import torch
    import fp8_layers
    x, state, _ = fp8_layers.decode(tokens=5, hidden=256, inner=384, experts=8, steps=3)
    g = torch.Generator(device="cuda").manual_seed(0)
    block = fp8_layers.ExpertBlock(256, 384, 8, 2, g)
    a = torch.randn(5, 256, device="cuda", generator=g).bfloat16()
    b = torch.zeros_like(a)
    for _ in range(3):
        a, b = block(a, b)
    torch.cuda.synchronize()
    assert torch.equal(a, x) and torch.equal(b, state)
    assert bool(torch.isfinite(x.float()).all()) and float(x.float().abs().max()) > 0
