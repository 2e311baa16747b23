"""The quantiser (sgemm_fp8_quantize): scales and codes equal, bit for bit, to the definition's
operations done one by one in numpy."""
import numpy as np
import pytest

import sgemm_row_major_gb300 as sg
from fp8_util import TINY, code_values, quantize_ref, round_codes, strided, values

GROUPS = [(1, 128), (128, 1), (128, 128)]
FAKE = 1 << 20


def make(rows, cols, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    x *= np.exp2(rng.integers(-12, 12, size=(1, cols))).astype(np.float32)
    return x


def check(x, block, fmt, pad=0, offset=0, dtype="float32"):
    import torch
    t = torch.from_numpy(x).to(getattr(torch, dtype))
    ref_s, ref_q = quantize_ref(t.float().numpy(), block, fmt)
    m = sg.quantize_fp8(strided(t, pad, offset), block, fmt)
    torch.cuda.synchronize()
    s, q = m.scale.cpu().numpy(), values(m)
    assert np.array_equal(s, ref_s), np.argwhere(s != ref_s)[:4]
    same = (q == ref_q) | (np.isnan(q) & np.isnan(ref_q))
    assert same.all(), (np.argwhere(~same)[:4], q[~same][:4], ref_q[~same][:4])


def test_rounding_reference_fixes_every_code():
    """The numpy rounding used below: every finite code is its own nearest, midpoints go to the even code."""
    for fmt in ("e4m3", "e5m2"):
        v = code_values(fmt)
        pos = v[:128][np.isfinite(v[:128])]
        assert np.array_equal(round_codes(pos, fmt), pos)
        mid = (pos[:-1] + pos[1:]) / 2
        assert np.array_equal(round_codes(mid, fmt), pos[np.arange(len(mid)) + (np.arange(len(mid)) % 2)])
    assert code_values("e4m3")[126] == 448 and code_values("e5m2")[123] == 57344


@pytest.mark.gpu
@pytest.mark.parametrize("block", GROUPS)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (127, 129), (128, 128), (257, 1000), (300, 130), (2000, 3)])
def test_equal_to_the_definition(block, fmt, dtype, rows, cols):
    check(make(rows, cols, rows + cols), block, fmt, dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("block", GROUPS)
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_strides_and_alignment(block, pad, offset, dtype):
    check(make(200, 328, 9), block, "e4m3", pad, offset, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("block", GROUPS)
def test_special_values(block):
    """NaN and infinities become NaN codes and do not count towards the scale; zeros, subnormals and the
    largest floats keep finite scales; ties go to even."""
    x = make(256, 384, 3)
    x[0, 0], x[1, 130], x[130, 5], x[131, 6] = np.nan, np.inf, -np.inf, np.nan
    x[2, :128] = 0.0
    x[3, :128] = np.float32(1e-42)
    x[4, 256:384] = np.float32(3e38)
    x[5, :128] = np.inf
    x[128:256, 128:256] = 0.0
    x[:, 300] = 0.0
    check(x, block, "e4m3")
    check(x, block, "e5m2")
    tie = np.ones((128, 128), np.float32) * 448.0  # scale 1: the codes' own midpoints
    v = code_values("e4m3")[:127]
    tie.reshape(-1)[:126] = (v[:-1] + v[1:]) / 2
    check(tie, (128, 128), "e4m3")


@pytest.mark.gpu
def test_every_bf16_value_of_a_group():
    """All finite BF16 values, one binade range per group: the conversion over its whole range."""
    bits = np.arange(1 << 16, dtype=np.uint32) << 16
    x = bits.view(np.float32).reshape(512, 128).copy()
    check(x, (1, 128), "e4m3")
    check(x, (1, 128), "e5m2")


@pytest.mark.gpu
def test_runs_on_the_given_stream_and_in_a_graph():
    import torch
    x = torch.from_numpy(make(300, 512, 4)).cuda()
    want = sg.quantize_fp8(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sg.quantize_fp8(x, stream=side)
    side.synchronize()
    assert torch.equal(got.data.view(torch.uint8), want.data.view(torch.uint8)) and torch.equal(got.scale, want.scale)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m = sg.quantize_fp8(x)
    x.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(m.scale, 2 * want.scale) and torch.equal(m.data.view(torch.uint8), want.data.view(torch.uint8))


@pytest.mark.gpu
def test_empty():
    import torch
    for shape in ((0, 5), (5, 0), (0, 0)):
        m = sg.quantize_fp8(torch.zeros(shape, device="cuda"))
        assert tuple(m.shape) == shape


@pytest.mark.gpu
def test_rows_without_a_stride_are_refused():
    """An expanded tensor's rows share memory: no leading dimension describes it."""
    import torch
    x = torch.zeros(1, 256, device="cuda").expand(5, 256)
    with pytest.raises(sg.SgemmError):
        sg.quantize_fp8(x)
    with pytest.raises(sg.SgemmError):
        sg.rmsnorm_fp8(x, torch.ones(256, device="cuda"))


def call(*a):
    from sgemm_row_major_gb300 import fp8
    return fp8._lib().sgemm_fp8_quantize(*a)


def test_refusals():
    """Invalid arguments return -(index) and launch nothing (the addresses are not memory)."""
    ok = [4, 256, FAKE, 0, 256, 0, 1, 128, FAKE, 256, FAKE, 2, None]
    for index, value in [(1, -1), (2, -1), (3, None), (3, FAKE + 2), (4, 2), (5, 255), (6, 2), (7, 2), (7, 0), (8, 64), (8, 1),
                         (9, None), (10, 255), (11, None), (11, FAKE + 1), (12, 1)]:
        bad = list(ok)
        bad[index - 1] = value
        assert call(*bad) == -index, (index, value)
    assert call(0, 256, None, 0, 256, 0, 1, 128, None, 256, None, 2, None) == 0


def test_python_refusals():
    import torch
    with pytest.raises(TypeError):
        sg.quantize_fp8(torch.zeros(4, 4))
    assert TINY == np.float32(2.0 ** -126)
