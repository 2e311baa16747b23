"""BF16 layers over very long sums."""
import math

import pytest

import sgemm_row_major_gb300 as sg


def test_gated_long_sums_have_a_tile_that_folds():
    """A gated tile of 128 columns takes whole sums alone: not of more than 16384 terms, chosen or forced."""
    from sgemm_row_major_gb300 import build
    build.build()
    try:
        for rows, cols in ((300, 700), (1000, 64), (4096, 8192)):
            for variant, tile in (("LINEAR_PAIR", 0), ("LINEAR_PAIR", 128), ("AUTO", 0)):
                sg.sgemm_linear_set_override(variant, tile)
                p = sg.sgemm_linear_plan(rows, cols, 16385, gated=True, sm_count=152)
                assert p["variant_name"] == "LINEAR_SHORT" or p["tile_n"] == 256
        sg.sgemm_linear_set_override("LINEAR_PAIR", 128)
        assert sg.sgemm_linear_plan(300, 700, 16384, gated=True, sm_count=152)["tile_n"] == 128
    finally:
        sg.sgemm_linear_set_override()


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [("AUTO", 0, 0), ("LINEAR_PAIR", 256, 1), ("LINEAR_PAIR", 128, 1), ("LINEAR_PAIR", 64, 1), ("LINEAR_PAIR", 64, 4),
                                    ("LINEAR_SHORT", 64, 2)], ids=str)
def test_long_sums_do_not_drift(kernel):
    """BF16 results of 2^20 terms of one sign, on average over 2^16 of them.  The tensor cores truncate what they add, and the more
    the larger the sum in one accumulator is: over 256 K tiles of 64 it comes out 7.5e-5 too small (measured), over 16384 6.6e-3.
    Allowed are 8.9e-5, a twentieth of BF16's smallest half step, and the rounding to BF16: at most 2^-8 either way, evenly spread
    where the results are spread evenly over a binade, so its mean over n of them has a deviation of 2^-8 / sqrt(3 n), of which six
    are counted.  A gated result has two such factors."""
    import torch
    n, K = 256, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(7)

    def spread(*shape):  # positive, rows with factors spread evenly over the logarithm of [1, 2)
        v = torch.rand(*shape, generator=g, device="cuda") + 0.5
        return (v * 2.0 ** torch.rand(shape[0], 1, generator=g, device="cuda")).bfloat16()

    tol = 8.9e-5 + 6 * 2.0 ** -8 / math.sqrt(3 * n * n)  # 1.4e-4
    off = lambda got, want: float(((got.double() - want) / want).mean())  # noqa: E731
    x, w, u = spread(n, K), spread(n, K) / K, spread(n, K) / K
    a, b = x.double() @ w.double().T, x.double() @ u.double().T
    sg.sgemm_linear_set_override(*kernel)
    try:
        y = sg.linear_bf16(x, w, save="bf16")
        h = sg.gated_bf16(x, w, u, None, save="bf16")
        dw = sg.linear_bf16_backward(x.T.contiguous(), w.T.contiguous(), None, dx=False).dweight
    finally:
        sg.sgemm_linear_set_override()
    got = {"y": off(y.y, a), "pre": off(y.pre, a), "gate": off(h.gate, a), "up": off(h.up, b), "dweight": off(dw, a), "h": off(h.h, a * b) / 2}
    assert all(abs(v) <= tol for v in got.values()), (tol, got)
    assert sg.sgemm_sync_status() == 0
