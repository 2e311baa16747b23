"""Values of the BF16 layers that their header speaks of: NaN and infinities through the activations, FP32 results of the longest
sums that it names."""
import math

import pytest

import sgemm_row_major_gb300 as sg
from test_linear import done, rand

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


@pytest.mark.parametrize("kernel", [("LINEAR_SHORT", 16, 1), ("LINEAR_PAIR", 64, 0), ("LINEAR_PAIR", 256, 0), ("LINEAR_PAIR", 64, 2)], ids=str)
def test_special_values(kernel):
    """NaN, the infinities and both zeros through every activation and its derivative (as a bias on a product of zeros)."""
    import torch
    values = torch.tensor([NAN, INF, -INF, 0.0, -0.0], device="cuda").bfloat16()
    x, w = torch.zeros(3, 256, device="cuda").bfloat16(), torch.zeros(5, 256, device="cuda").bfloat16()
    half = {"relu": 0.0, "silu": 0.5, "gelu": 0.5, "gelu_tanh": 0.5}
    sg.sgemm_linear_set_override(*kernel)
    try:
        for activation in (None, *half):
            for dtype in (torch.bfloat16, torch.float32):
                got = sg.linear_bf16(x, w, values, activation, save="bf16", out_dtype=dtype)
                low = {None: -INF, "relu": 0.0}.get(activation, NAN)
                for out, want in ((got.y, [NAN, INF, low, 0.0, 0.0]), (got.pre, [NAN, INF, -INF, 0.0, 0.0])):
                    assert torch.equal(out.float().nan_to_num(7.0, 8.0, 9.0), torch.tensor([want] * 3, device="cuda").nan_to_num(7.0, 8.0, 9.0)), activation
            if activation:
                pre = values[None].contiguous()
                d = sg.linear_bf16_backward(torch.ones_like(pre), None, None, pre, activation, dx=False, dweight=False, dbias=True).dbias.tolist()
                # at 0: Phi's polynomial is 4.4e-7 of itself off (linear_common.cuh), 2.2e-7 at 1/2; the bound of linear_util.py is 32 u
                assert math.isnan(d[0]) and d[1:3] == [1.0, 0.0] and all(abs(v - half[activation]) <= 32 * 2.0 ** -24 for v in d[3:]), activation
    finally:
        sg.sgemm_linear_set_override()
    done()


@pytest.mark.parametrize("kernel", [("AUTO", 0, 0), ("LINEAR_PAIR", 256, 1), ("LINEAR_PAIR", 128, 0), ("LINEAR_SHORT", 64, 1)], ids=str)
def test_fp32_values_of_16384_terms(kernel):
    """Random sums of 16384 terms, FP32 outputs and the scales of 8-bit values: within 1e-6 in norm, as the header says."""
    import torch
    T, I, O = 300, 16384, 256
    x, w, u = rand(1, T, I), rand(2, O, I, std=I ** -0.5), rand(3, O, I, std=I ** -0.5)
    pre = x.double() @ w.double().T
    scale = pre.abs().view(T, -1, 128).amax(2) / 448
    off = lambda got, want: float((got.double() - want).norm() / want.norm())  # noqa: E731
    sg.sgemm_linear_set_override(*kernel)
    try:
        got = {"y": off(sg.linear_bf16(x, w, out_dtype=torch.float32).y, pre), "scale": off(sg.linear_bf16(x, w, save="fp8").pre.scale, scale),
               "gate": off(sg.gated_bf16(x, w, u, save="fp8").gate.scale, scale),
               "dweight": off(sg.linear_bf16_backward(x.T.contiguous(), w.T.contiguous(), None, dx=False, dweight_dtype=torch.float32).dweight, pre)}
    finally:
        sg.sgemm_linear_set_override()
    assert max(got.values()) <= 1e-6, got
    done()
