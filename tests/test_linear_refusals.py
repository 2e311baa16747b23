"""What the entry points of the BF16 layers refuse, and what their planner chooses: no GPU."""
import ctypes

import pytest

import sgemm_row_major_gb300 as sg
from sgemm_row_major_gb300 import fp8, linear
from test_fp8_python import Stand

FAKE = 1 << 20  # an aligned device address (never dereferenced here)


@pytest.fixture(scope="module")
def lib():
    from sgemm_row_major_gb300 import build
    build.build()
    return linear._lib()


def kept(data=FAKE, ld=16, scale=None, lds=1):
    return linear.KeptStruct(data, ld, scale, lds)


def refused(f, good, cases, empty=()):
    """Each change of the good arguments (1-based index, value) gives its status before anything is launched."""
    for status, changes in cases:
        args = list(good)
        for at, value in changes.items():
            args[at - 1] = value
        assert f(*args) == status, (status, changes)
        assert "invalid argument" in sg.sgemm_status_string(status) or status > 0
    for changes in empty:
        args = list(good)
        for at, value in changes.items():
            args[at - 1] = value
        assert f(*args) == 0, changes


def test_layer_arguments(lib):
    # tokens, inputs, outputs, X, ldx, W, ldw, bias, act, R, ldr, kept, Y, ldy, type, stream
    good = (4, 8, 16, FAKE, 8, FAKE, 8, FAKE, 2, FAKE, 16, kept(), FAKE, 16, 1, None)
    refused(lib.sgemm_linear, good, [
        (-1, {1: -1}), (-2, {2: -1}), (-3, {3: -1}), (-4, {4: None}), (-4, {4: FAKE + 1}), (-5, {5: 7}), (-6, {6: None}), (-7, {7: 7}),
        (-8, {8: FAKE + 1}), (-9, {9: 5}), (-9, {9: -1}), (-10, {10: FAKE + 1}), (-11, {11: 15}), (-12, {12: kept(None)}), (-12, {12: kept(ld=15)}),
        (-12, {12: kept(FAKE + 1)}), (-12, {12: kept(scale=FAKE + 2)}), (-12, {12: kept(scale=FAKE, lds=0)}), (-13, {13: None}), (-13, {13: FAKE + 1}),
        (-13, {13: FAKE + 2, 15: 0}), (-13, {15: 0}), (-14, {14: 15}), (-14, {14: 24}), (-15, {15: 2}),
        (4, {1: (1 << 31) - 1}), (4, {2: 1 << 31, 5: 1 << 31, 7: 1 << 31}), (4, {5: 1 << 31}),
    ], empty=[{1: 0, 4: None, 13: None}, {3: 0, 6: None, 13: None}])


def test_gated_arguments(lib):
    # tokens, inputs, outputs, X, ldx, gate, ldg, up, ldu, act, kept_gate, kept_up, H, ldh, stream
    good = (4, 8, 16, FAKE, 8, FAKE, 8, FAKE, 8, 2, kept(), kept(), FAKE, 16, None)
    refused(lib.sgemm_gated, good, [
        (-1, {1: -1}), (-2, {2: -1}), (-3, {3: -1}), (-4, {4: None}), (-5, {5: 7}), (-6, {6: None}), (-7, {7: 7}), (-8, {8: None}), (-9, {9: 7}),
        (-10, {10: 9}), (-11, {11: kept(None)}), (-12, {12: None}), (-12, {11: None}), (-12, {12: kept(scale=FAKE)}), (-12, {12: kept(ld=15)}),
        (-13, {13: None}), (-13, {13: FAKE + 1}), (-14, {14: 15}), (4, {14: 1 << 31}),
    ], empty=[{1: 0, 4: None, 13: None}, {3: 0, 13: None}])


def test_layer_gradient_arguments(lib):
    # tokens, inputs, outputs, dY, lddy, X, W, ldw, act, kept, dX, lddx, dW, lddw, dw_type, dbias, stream
    good = (4, 8, 16, FAKE, 16, kept(ld=8), FAKE, 8, 2, kept(), FAKE, 8, FAKE, 8, 1, FAKE, None)
    refused(lib.sgemm_linear_backward, good, [
        (-1, {1: -1}), (-2, {2: -1}), (-3, {3: -1}), (-4, {4: None}), (-5, {5: 15}), (-6, {6: None}), (-6, {6: kept(ld=7)}), (-7, {7: None}), (-8, {8: 7}),
        (-9, {9: 5}), (-10, {10: None}), (-10, {10: kept(None)}), (-11, {11: FAKE + 1}), (-12, {12: 7}), (-13, {13: FAKE + 1}), (-13, {13: FAKE + 2, 15: 0}),
        (-14, {14: 7}), (-15, {15: 2}), (-16, {16: FAKE + 2}), (4, {1: 1 << 31}), (4, {12: 1 << 31}),
    ], empty=[{11: None, 13: None, 16: None}, {1: 0, 4: None, 6: kept(None, ld=8), 10: kept(None), 13: None, 16: None},
              {11: None, 13: None, 16: None, 6: None, 7: None, 10: kept()}])


def test_gated_gradient_arguments(lib):
    # tokens, inputs, outputs, dH, lddh, X, gate, ldg, up, ldu, act, kept_gate, kept_up, dX, lddx, dG, lddg, dU, lddu, dw_type, H, ldh, stream
    good = (4, 8, 16, FAKE, 16, kept(ld=8), FAKE, 8, FAKE, 8, 2, kept(), kept(), FAKE, 8, FAKE, 8, FAKE, 8, 1, FAKE, 16, None)
    refused(lib.sgemm_gated_backward, good, [
        (-1, {1: -1}), (-2, {2: -1}), (-3, {3: -1}), (-4, {4: None}), (-5, {5: 15}), (-6, {6: None}), (-7, {7: None}), (-8, {8: 7}), (-9, {9: None}),
        (-10, {10: 7}), (-11, {11: 5}), (-12, {12: None}), (-13, {13: None}), (-13, {13: kept(scale=FAKE)}), (-14, {14: FAKE + 1}), (-15, {15: 7}),
        (-16, {16: FAKE + 1}), (-17, {17: 7}), (-18, {18: None}), (-18, {16: None}), (-19, {19: 7}), (-20, {20: 2}), (-21, {21: FAKE + 1}), (-22, {22: 15}),
        (4, {17: 1 << 31}),
    ], empty=[{14: None, 16: None, 18: None, 21: None}])


def test_planner(lib):
    """Few tokens on the short-side kernel with K shared, many on CTA pairs; kept 8-bit groups on tiles that hold them."""
    p = sg.sgemm_linear_plan(1, 4096, 4096, sm_count=152)
    assert p["variant_name"] == "LINEAR_SHORT" and p["tile_n"] == 16 and p["split_k"] > 1 and p["grid_x"] == 32 * p["split_k"]
    p = sg.sgemm_linear_plan(8192, 16384, 4096, sm_count=152)
    assert p["variant_name"] == "LINEAR_PAIR" and p["tile_n"] == 256 and p["grid_x"] == 152 and p["stages"] == 5
    for rows in (1, 40, 300, 2000):
        for cols in (60, 128, 700, 5000):
            p = sg.sgemm_linear_plan(rows, cols, 640, gated=True, kept8=True, sm_count=152)
            assert p["variant_name"] == "LINEAR_SHORT" and p["tile_n"] <= 64 or p["tile_n"] == 256
            p = sg.sgemm_linear_plan(rows, cols, 640, kept8=True, sm_count=152)
            assert p["variant_name"] == "LINEAR_SHORT" or p["tile_n"] >= 128
            assert p["smem_bytes"] <= 232448 and 1 <= p["stages"] <= 12
    for bad, status in (((0, 8, 8), -1), ((8, 0, 8), -2), ((8, 8, 0), -3), ((1 << 31, 8, 8), 4)):
        with pytest.raises(sg.SgemmError) as e:
            sg.sgemm_linear_plan(*bad, sm_count=152)
        assert e.value.status == status
    assert lib.sgemm_linear_plan(8, 8, 8, 0, 0, 152, None) == -7


def test_override(lib):
    try:
        for v, t, k in ((0, 0, 0), (40, 256, 0), (40, 0, 0), (41, 16, 8), (41, 128, 1), (40, 64, 2), (40, 0, 32)):
            assert lib.sgemm_linear_set_override(v, t, k) == 0
        for args, status in (((32, 0, 0), -1), ((40, 16, 0), -2), ((41, 256, 0), -2), ((0, 64, 0), -2), ((40, 64, 33), -3), ((40, 64, -1), -3), ((0, 0, 2), -3), ((41, 16, 3), -3)):
            assert lib.sgemm_linear_set_override(*args) == status
        sg.sgemm_linear_set_override("LINEAR_SHORT", 32, 2)
        p = sg.sgemm_linear_plan(1000, 1000, 1000, sm_count=152)
        assert (p["variant_name"], p["tile_n"], p["split_k"]) == ("LINEAR_SHORT", 32, 2)
        sg.sgemm_linear_set_override("LINEAR_PAIR", 64)  # (too narrow for a gated tile: the planner's own)
        assert sg.sgemm_linear_plan(1000, 1000, 1000, gated=True, sm_count=152)["tile_n"] in (128, 256)
        sg.sgemm_linear_set_override("LINEAR_SHORT", 128)
        assert sg.sgemm_linear_plan(1000, 1000, 1000, gated=True, sm_count=152)["tile_n"] < 128
    finally:
        sg.sgemm_linear_set_override()


@pytest.fixture
def on_device_0(monkeypatch):
    """Device 0 is current; nothing is allocated and the library is not called."""
    linear._lib()
    monkeypatch.setattr(fp8, "_current_device", lambda: 0)

    def never(*a, **k):
        raise AssertionError("the call got past its checks")
    for module in (fp8, linear):
        monkeypatch.setattr(module, "_empty", never)
        monkeypatch.setattr(module, "_new_matrix", never)
    monkeypatch.setattr(fp8, "_raw_stream", never)


class Columns(Stand):
    """A matrix whose columns are contiguous."""

    def stride(self, i=None):
        return (1, self.shape[0])


def matrix8(rows, cols, device=0, block=(1, 128), fmt=None):
    import torch
    return sg.Fp8Matrix(Stand((rows, cols), fmt or torch.float8_e4m3fn, device), Stand((-(-rows // block[0]), -(-cols // block[1])), torch.float32, device), block)


def test_tensors_of_different_devices_are_refused(on_device_0):
    import torch
    bf = torch.bfloat16
    S = lambda shape, dev: Stand(shape, bf, dev)  # noqa: E731
    calls = [
        (5, lambda x, w, b, r, o: sg.linear_bf16(S((4, 8), x), S((16, 8), w), S((16,), b), None, S((4, 16), r), out=S((4, 16), o))),
        (4, lambda x, g, u, o: sg.gated_bf16(S((4, 8), x), S((16, 8), g), S((16, 8), u), out=S((4, 16), o))),
        (4, lambda d, x, w, p: sg.linear_bf16_backward(S((4, 16), d), S((4, 8), x), S((16, 8), w), S((4, 16), p), "gelu")),
        (4, lambda d, x, w, p: sg.linear_bf16_backward(S((4, 16), d), matrix8(4, 8, x), S((16, 8), w), matrix8(4, 16, p), "gelu")),
        (6, lambda d, x, g, u, a, b: sg.gated_bf16_backward(S((4, 16), d), S((4, 8), x), S((16, 8), g), S((16, 8), u), S((4, 16), a), S((4, 16), b))),
    ]
    for n, call in calls:
        for other in range(n):
            with pytest.raises(ValueError, match="device"):
                call(*(int(i == other) for i in range(n)))
        with pytest.raises(ValueError, match="current device"):
            call(*(1 for _ in range(n)))
        with pytest.raises(AssertionError, match="past its checks"):
            call(*(0 for _ in range(n)))


def test_layer_refusals(on_device_0):
    """Shapes, types, orders and options that do not fit."""
    import torch
    bf, f32 = torch.bfloat16, torch.float32
    S = Stand

    def call(error, **kw):
        a = dict(x=S((4, 8), bf), weight=S((16, 8), bf), bias=S((16,), bf), activation="gelu", residual=S((4, 16), bf))
        a.update(kw)
        with pytest.raises(error):
            sg.linear_bf16(**a)
    call(AssertionError)
    call(TypeError, x=S((4, 8), f32))
    call(TypeError, weight=S((16, 8), torch.float16))
    call(TypeError, x=S((2, 4, 8), bf))
    call(TypeError, x=Columns((4, 8), bf))
    call(ValueError, weight=S((16, 9), bf))
    call(ValueError, bias=S((15,), bf))
    call(TypeError, bias=S((16,), f32))
    call(ValueError, residual=S((4, 15), bf))
    call(TypeError, residual=S((4, 16), f32))
    call(ValueError, activation="tanh")
    call(ValueError, activation=["gelu"])
    call(ValueError, save="e5m2")
    call(ValueError, out=S((4, 15), bf))
    call(TypeError, out=S((4, 16), torch.float16))
    call(TypeError, out=S((4, 16), bf), out_dtype=f32)
    call(TypeError, out_dtype=torch.float16)


def test_gated_refusals(on_device_0):
    import torch
    bf = torch.bfloat16
    S = Stand

    def call(error, **kw):
        a = dict(x=S((4, 8), bf), gate=S((16, 8), bf), up=S((16, 8), bf))
        a.update(kw)
        with pytest.raises(error):
            sg.gated_bf16(**a)
    call(AssertionError)
    call(ValueError, up=S((15, 8), bf))
    call(ValueError, gate=S((16, 7), bf))
    call(TypeError, up=S((16, 8), torch.float32))
    call(ValueError, activation="swish")
    call(ValueError, save="fp4")
    call(TypeError, out=S((4, 16), torch.float32))


def test_gradient_refusals(on_device_0):
    import torch
    bf, f32 = torch.bfloat16, torch.float32
    S = Stand

    def one(error, **kw):
        a = dict(dy=S((4, 16), bf), x=S((4, 8), bf), weight=S((16, 8), bf), pre=S((4, 16), bf), activation="silu")
        a.update(kw)
        with pytest.raises(error):
            sg.linear_bf16_backward(**a)
    one(AssertionError)
    one(ValueError, pre=None)
    one(ValueError, pre=S((4, 15), bf))
    one(TypeError, pre=S((4, 16), f32))
    one(ValueError, pre=matrix8(4, 15))
    one(ValueError, pre=matrix8(4, 16, block=(128, 128)))
    one(ValueError, pre=matrix8(4, 16, fmt=torch.float8_e5m2))
    one(ValueError, x=matrix8(5, 8))
    one(ValueError, x=S((4, 9), bf))
    one(ValueError, weight=S((15, 8), bf))
    one(TypeError, dy=S((4, 16), f32))
    one(ValueError, activation="sigmoid")

    def two(error, **kw):
        a = dict(dh=S((4, 16), bf), x=S((4, 8), bf), gate=S((16, 8), bf), up=S((16, 8), bf), gate_pre=S((4, 16), bf), up_pre=S((4, 16), bf))
        a.update(kw)
        with pytest.raises(error):
            sg.gated_bf16_backward(**a)
    two(AssertionError)
    two(TypeError, up_pre=matrix8(4, 16))
    two(ValueError, gate_pre=S((4, 17), bf))
    two(ValueError, up=S((16, 9), bf))
    two(ValueError, x=S((3, 8), bf))
    two(ValueError, gate_pre=matrix8(4, 16, block=(128, 1)), up_pre=matrix8(4, 16))


def test_structure_sizes():
    assert ctypes.sizeof(linear.KeptStruct) == 32
