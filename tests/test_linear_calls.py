"""Calls of the BF16 layers that are refused, by the C entry points and in Python: no GPU."""
import pytest

import sgemm_row_major_gb300 as sg
from test_linear_refusals import FAKE, Stand, kept, lib, matrix8, on_device_0, refused  # noqa: F401 (fixtures)

WIDE = 1 << 31  # a row stride that is not supported


def test_kept_rows_too_far_apart(lib):  # noqa: F811
    """A kept matrix whose row stride is too large is as unsupported as any other, and one that is not read is not looked at."""
    unsupported = sg.STATUS["ERR_UNSUPPORTED"]
    for scale in (None, FAKE):
        far, near = kept(ld=WIDE, scale=scale), kept(ld=16, scale=scale)
        layer = (4, 8, 16, FAKE, 8, FAKE, 8, FAKE, 2, FAKE, 16, near, FAKE, 16, 1, None)
        refused(lib.sgemm_linear, layer, [(unsupported, {12: far})], empty=[{1: 0, 12: far}])
        gated = (4, 8, 16, FAKE, 8, FAKE, 8, FAKE, 8, 2, near, near, FAKE, 16, None)
        refused(lib.sgemm_gated, gated, [(unsupported, {11: far}), (unsupported, {12: far})])
        grad = (4, 8, 16, FAKE, 16, kept(ld=8, scale=scale), FAKE, 8, 2, near, FAKE, 8, FAKE, 8, 1, FAKE, None)
        refused(lib.sgemm_linear_backward, grad, [(unsupported, {6: far}), (unsupported, {10: far}), (-6, {6: kept(ld=7, scale=scale)})],
                empty=[{6: far, 10: far, 9: 0, 11: None, 13: None, 16: None}])
        grad = (4, 8, 16, FAKE, 16, kept(ld=8, scale=scale), FAKE, 8, FAKE, 8, 2, near, near, FAKE, 8, FAKE, 8, FAKE, 8, 1, FAKE, 16, None)
        refused(lib.sgemm_gated_backward, grad, [(unsupported, {6: far}), (unsupported, {12: far}), (unsupported, {13: far}), (-12, {12: kept(ld=15, scale=scale)})],
                empty=[{6: far, 14: None, 16: None, 18: None, 21: None}])


def no_matrices():
    """What is no matrix of BF16 values: nothing, a number, a list, a vector, and one of each wrong type."""
    import numpy as np
    import torch
    return [None, 3, [[1.0]], np.zeros((4, 8), np.float32), Stand((8,), torch.bfloat16), Stand((4, 8), torch.float32)]


def test_operands_that_are_no_matrices(on_device_0):  # noqa: F811
    """A TypeError that names the operand, whichever gradients are wanted."""
    import torch
    bf = torch.bfloat16
    layer = dict(x=Stand((4, 8), bf), weight=Stand((16, 8), bf), bias=Stand((16,), bf), residual=Stand((4, 16), bf), out=Stand((4, 16), bf))
    gated = dict(x=Stand((4, 8), bf), gate=Stand((16, 8), bf), up=Stand((16, 8), bf), out=Stand((4, 16), bf))
    grad = dict(dy=Stand((4, 16), bf), x=Stand((4, 8), bf), weight=Stand((16, 8), bf), pre=Stand((4, 16), bf), activation="silu")
    gated_grad = dict(dh=Stand((4, 16), bf), x=Stand((4, 8), bf), gate=Stand((16, 8), bf), up=Stand((16, 8), bf), gate_pre=Stand((4, 16), bf),
                      up_pre=Stand((4, 16), bf))
    optional = ("bias", "residual", "out", "pre")
    takes8 = ("x", "pre", "gate_pre", "up_pre")
    calls = [(sg.linear_bf16, layer, {}, ()), (sg.gated_bf16, gated, {}, ()),
             (sg.linear_bf16_backward, grad, {}, ()), (sg.linear_bf16_backward, grad, dict(dx=False), ("weight",)),
             (sg.linear_bf16_backward, grad, dict(dweight=False), ("x",)),
             (sg.gated_bf16_backward, gated_grad, {}, ()), (sg.gated_bf16_backward, gated_grad, dict(dx=False), ("gate", "up")),
             (sg.gated_bf16_backward, gated_grad, dict(dweights=False), ("x",))]
    for f, good, wanted, unread in calls:
        with pytest.raises(AssertionError, match="past its checks"):
            f(**good, **wanted)
        for name, value in good.items():
            if not hasattr(value, "shape"):
                continue
            for bad in no_matrices() + ([] if name in takes8 and "backward" in f.__name__ else [matrix8(*value.shape) if len(value.shape) == 2 else 1]):
                if bad is None and name in optional or name == "out" and getattr(bad, "dtype", None) is torch.float32 or name == "bias" and getattr(bad, "shape", None) == (8,):
                    continue
                if name in unread:
                    with pytest.raises(AssertionError, match="past its checks"):
                        f(**{**good, name: bad}, **wanted)
                    continue
                with pytest.raises(TypeError, match=f"^{name} "):
                    f(**{**good, name: bad}, **wanted)
