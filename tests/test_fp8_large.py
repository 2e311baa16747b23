"""The 8-bit operators on operands whose offsets pass 2^31 elements: the results of the same values stored closely, bit
for bit.  (The product: test_fp8_product.py, test_offsets_past_32_bits.)"""
import pytest

import sgemm_row_major_gb300 as sg

ROWS, COLS, LD = 60000, 200, 40000  # the last rows begin 2.4e9 elements from the first


def far(x, ld=LD):
    """x's values in rows `ld` elements apart."""
    import torch
    v = torch.empty(x.shape[0] * ld, dtype=x.dtype, device="cuda").view(x.shape[0], ld)[:, : x.shape[1]]
    v.copy_(x)
    return v


def same(a, b):
    import torch
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.fixture(autouse=True)
def free():
    yield
    import torch
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("cols", [COLS, COLS - 1])
def test_rows_far_apart(dtype, cols):
    import torch
    from sgemm_row_major_gb300 import fp8
    t = getattr(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = (torch.randn(ROWS, cols, generator=g, device="cuda").to(t) for _ in range(2))
    w = torch.ones(cols, dtype=t, device="cuda")
    a, b = far(x), far(dy)
    for block in fp8.GROUPS:
        want, got = sg.quantize_fp8(x, block), sg.quantize_fp8(a, block)
        assert same(got.data, want.data) and same(got.scale, want.scale)
    want, got = sg.rmsnorm_fp8(x, w, 1e-6, dy, y=True), sg.rmsnorm_fp8(a, w, 1e-6, b, y=True)
    assert same(got.q.data, want.q.data) and same(got.h, want.h) and same(got.y, want.y) and same(got.rstd, want.rstd)
    if cols % 8 == 0:  # (another alignment of the rows takes another kernel)
        wdx, wdw = sg.rmsnorm_fp8_backward(dy, x, w, want.rstd)
        dx, dw = sg.rmsnorm_fp8_backward(b, a, w, want.rstd)
        assert same(dx, wdx) and same(dw, wdw)
        # outputs far apart: dX over dY
        st = fp8._lib().sgemm_fp8_rmsnorm_backward(ROWS, cols, fp8._TYPES[t], b.data_ptr(), LD, a.data_ptr(), LD, w.data_ptr(), want.rstd.data_ptr(),
                                                   None, 0, b.data_ptr(), LD, dw.data_ptr(), None)
        torch.cuda.synchronize()
        assert st == 0 and same(b, wdx) and same(dw, wdw)


@pytest.mark.gpu
def test_experts_far_apart():
    import torch
    E, H, I, T, gap = 4, 256, 144, 20, 1 << 30
    g = torch.Generator(device="cuda").manual_seed(4)

    def stack(rows, cols):
        codes = torch.randint(0, 0x50, (E, rows, cols), generator=g, device="cuda", dtype=torch.uint8)
        wide = torch.empty(E * gap, dtype=torch.uint8, device="cuda").as_strided((E, rows, cols), (gap, cols, 1))
        wide.copy_(codes)
        scale = torch.rand(E, -(-rows // 128), -(-cols // 128), generator=g, device="cuda")
        return (codes.view(torch.float8_e4m3fn), scale), (wide.view(torch.float8_e4m3fn), scale)
    pairs = [stack(I, H), stack(I, H), stack(H, I)]
    x, logits = sg.quantize_fp8(torch.randn(T, H, generator=g, device="cuda")), torch.randn(T, E, generator=g, device="cuda")
    want = sg.moe_fp8(x, logits, 2, *(p[0] for p in pairs))
    y = far(torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), 1 << 27)  # the last rows 2.5e9 elements from the first
    assert same(sg.moe_fp8(x, logits, 2, *(p[1] for p in pairs), out=y), want)
