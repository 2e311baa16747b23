"""What the Python entry points of the 8-bit operators refuse or keep apart from their operands' values."""
import pytest

import sgemm_row_major_gb300 as sg
from sgemm_row_major_gb300 import fp8


class Stand:
    """What the entry points look at of a CUDA tensor, without a GPU."""

    is_cuda = True

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self.device = tuple(shape), dtype, device

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s, n = [], 1
        for d in reversed(self.shape):
            s.insert(0, n)
            n *= d
        return tuple(s) if i is None else s[i]

    def get_device(self):
        return self.device

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def on_device_0(monkeypatch):
    """Device 0 is current; nothing is allocated and the library is not called."""
    fp8._lib()
    monkeypatch.setattr(fp8, "_current_device", lambda: 0)

    def never(*a, **k):
        raise AssertionError("the call got past its checks")
    monkeypatch.setattr(fp8, "_empty", never)
    monkeypatch.setattr(fp8, "_raw_stream", never)


def test_tensors_of_different_devices_are_refused(on_device_0):
    """Each operand in turn on another device than the rest, and all of them on one that is not current."""
    import torch
    bf, f32, e4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

    def matrix(rows, cols, block, dev):
        return sg.Fp8Matrix(Stand((rows, cols), e4, dev), Stand((-(-rows // block[0]), -(-cols // block[1])), f32, dev), block)

    def experts(rows, cols, dev, scale_dev):
        return Stand((4, rows, cols), e4, dev), Stand((4, -(-rows // 128), -(-cols // 128)), f32, scale_dev)

    calls = [
        (1, lambda x: sg.quantize_fp8(Stand((4, 256), bf, x))),
        (4, lambda a, b, c, d: sg.matmul_fp8(matrix(8, 256, (1, 128), a), matrix(16, 256, (128, 128), b), Stand((8, 16), f32, c),
                                             transB="T", beta=1.0, out=Stand((8, 16), f32, d))),
        (3, lambda x, w, r: sg.rmsnorm_fp8(Stand((4, 256), bf, x), Stand((256,), bf, w), 1e-6, Stand((4, 256), bf, r))),
        (5, lambda dy, h, w, s, dh: sg.rmsnorm_fp8_backward(Stand((4, 256), bf, dy), Stand((4, 256), bf, h), Stand((256,), bf, w),
                                                            Stand((4,), f32, s), Stand((4, 256), bf, dh))),
        (9, lambda x, l, g, gs, u, us, d, ds, y: sg.moe_fp8(matrix(2, 256, (1, 128), x), Stand((2, 4), f32, l), 2, experts(128, 256, g, gs),
                                                            experts(128, 256, u, us), experts(256, 128, d, ds), out=Stand((2, 256), bf, y))),
    ]
    for n, call in calls:
        for other in range(n):
            with pytest.raises(ValueError, match="device"):
                call(*(int(i == other) for i in range(n)))
        with pytest.raises(ValueError, match="current device"):
            call(*(1 for _ in range(n)))
        with pytest.raises(AssertionError, match="past its checks"):
            call(*(0 for _ in range(n)))
    with pytest.raises(ValueError, match="scale on cuda:1"):
        sg.Fp8Matrix(Stand((8, 256), e4, 0), Stand((8, 2), f32, 1))


def test_a_stream_of_another_device_is_refused(on_device_0):
    import torch

    class Stream:
        cuda_stream = 77
        device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream"):
        sg.quantize_fp8(Stand((4, 256), torch.bfloat16), stream=Stream())


def test_a_matrix_attributes_are_fixed():
    """Codes or scales put in their place would not be the ones a call reads."""
    import torch
    fp8._lib()
    m = sg.Fp8Matrix(Stand((8, 256), torch.float8_e4m3fn), Stand((8, 2), torch.float32))
    for name in ("data", "scale", "block", "shape"):
        with pytest.raises(AttributeError):
            setattr(m, name, getattr(m, name))


@pytest.mark.gpu
def test_a_matrix_follows_its_tensors_memory():
    """A tensor whose memory was exchanged after the matrix was made is read where it is now; another shape is refused."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w = (torch.randn(n, 256, generator=g, device="cuda") for n in (8, 128))
    a, b = sg.quantize_fp8(x), sg.quantize_fp8(w, (128, 128))
    want = sg.matmul_fp8(a, b, transB="T")
    a.scale.data = a.scale * 2.0
    assert torch.equal(sg.matmul_fp8(a, b, transB="T"), 2.0 * want)
    b.data.data = b.data.view(torch.uint8).clone().bitwise_xor_(0x80).view(torch.float8_e4m3fn)
    assert torch.equal(sg.matmul_fp8(a, b, transB="T"), -2.0 * want)
    logits = torch.zeros(8, 2, device="cuda")
    up = torch.stack([b.data.view(torch.uint8)] * 2).view(torch.float8_e4m3fn), torch.stack([b.scale] * 2)
    d = sg.quantize_fp8(w.T.contiguous(), (128, 128))
    down = torch.stack([d.data.view(torch.uint8)] * 2).view(torch.float8_e4m3fn), torch.stack([d.scale] * 2)
    y = sg.moe_fp8(a, logits, 1, up, up, down)
    fresh = sg.Fp8Matrix(a.data.clone(), a.scale.clone())
    a.data.data = fresh.data.clone()
    a.data.view(torch.uint8).zero_()
    assert not torch.equal(sg.moe_fp8(a, logits, 1, up, up, down), y) and torch.equal(sg.moe_fp8(fresh, logits, 1, up, up, down), y)
    a.data.data = torch.zeros(4, 256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        sg.matmul_fp8(a, b, transB="T")


def test_experts_refusals(on_device_0):
    """Weights of another shape, type or order than the layer's."""
    import torch
    f32, e4 = torch.float32, torch.float8_e4m3fn
    x = sg.Fp8Matrix(Stand((2, 256), e4), Stand((2, 2), f32))

    def call(error, **kw):
        w = dict(gate=(Stand((4, 128, 256), e4), Stand((4, 1, 2), f32)), up=(Stand((4, 128, 256), e4), Stand((4, 1, 2), f32)),
                 down=(Stand((4, 256, 128), e4), Stand((4, 2, 1), f32)))
        w.update(kw)
        with pytest.raises(error):
            sg.moe_fp8(x, Stand((2, 4), f32), 2, w["gate"], w["up"], w["down"])

    class Columns(Stand):
        def stride(self, i=None):
            return (self.shape[1] * self.shape[2], 1, self.shape[1])
    good = Stand((4, 1, 2), f32)
    call(AssertionError)
    call(TypeError, up=(Stand((4 * 128, 256), e4), good))
    call(TypeError, up=(Stand((4, 128, 256), torch.float8_e5m2), good))
    call(TypeError, up=(Stand((4, 128, 256), e4), Stand((4, 1, 2), torch.bfloat16)))
    call(TypeError, up=(Columns((4, 128, 256), e4), good))
    call(ValueError, up=(Stand((4, 256, 256), e4), good))
    call(ValueError, up=(Stand((4, 128, 256), e4), Stand((4, 2, 2), f32)))
    call(ValueError, down=(Stand((4, 128, 256), e4), good))


def test_a_matrix_of_another_shape_stays_refused(on_device_0):
    """Memory and shape of a matrix's tensor exchanged: every call is refused, not only the first."""
    import torch
    a = sg.Fp8Matrix(Stand((8, 256), torch.float8_e4m3fn), Stand((8, 2), torch.float32))
    b = sg.Fp8Matrix(Stand((16, 256), torch.float8_e4m3fn), Stand((1, 2), torch.float32), (128, 128))
    a.data.shape, a.data.data_ptr = (8, 128), lambda: 1 << 21
    a.scale.shape = (8, 1)
    for _ in range(2):
        with pytest.raises(ValueError, match="had shape"):
            sg.matmul_fp8(a, b, transB="T")
    assert tuple(a.shape) == (8, 256)
