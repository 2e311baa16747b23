"""The operators on BF16 layers of libsgemm (C ABI in include/sgemm_linear.h): argument marshalling only.

``linear_bf16`` is a layer's product with bias, activation and residual, ``gated_bf16`` the first half of a gated
feed-forward block, both with their gradients.  What the backward pass needs of the values before the activation is
kept as BF16 or as an ``Fp8Matrix`` with groups of (1, 128).  Inputs are 2-D bfloat16 tensors with contiguous rows at any
alignment.  Outputs that a call allocates belong to the stream it runs on; their rows start at multiples of 8 elements (16
of codes), so where the width is not one they are not contiguous.  A call's tensors are on one device, which is the current
one (ValueError otherwise).
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

from . import PlanStruct, SgemmError, fp8
from .fp8 import ROW, Fp8Matrix, _empty, _new_matrix, _on, _rows

ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
VARIANTS = {0: "AUTO", 40: "LINEAR_PAIR", 41: "LINEAR_SHORT"}
KEEP = (None, "bf16", "fp8")


class KeptStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("scale", ctypes.c_void_p), ("lds", ctypes.c_int64)]


_declared = None  # the compiled library whose signatures are set
_bf16 = _f32 = None


def _declare(lib):
    """C signatures of this file's entry points."""
    i64, vp, ci, kp = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(KeptStruct)
    for name, args in {
        "sgemm_linear": [i64, i64, i64, vp, i64, vp, i64, vp, ci, vp, i64, kp, vp, i64, ci, vp],
        "sgemm_linear_backward": [i64, i64, i64, vp, i64, kp, vp, i64, ci, kp, vp, i64, vp, i64, ci, vp, vp],
        "sgemm_gated": [i64, i64, i64, vp, i64, vp, i64, vp, i64, ci, kp, kp, vp, i64, vp],
        "sgemm_gated_backward": [i64, i64, i64, vp, i64, kp, vp, i64, vp, i64, ci, kp, kp, vp, i64, vp, i64, vp, i64, ci, vp, i64, vp],
        "sgemm_linear_plan": [i64, i64, i64, ci, ci, ci, ctypes.POINTER(PlanStruct)],
        "sgemm_linear_set_override": [ci, ci, ci],
    }.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = ci, args
    return lib


def _lib():
    global _declared, _bf16, _f32
    lib = fp8._lib()
    if lib is not _declared:
        _declared = _declare(lib)
        _bf16, _f32 = fp8._T.bfloat16, fp8._T.float32
    return lib


def _no_tensor(x, name):
    return TypeError(f"{name} must be a tensor, got {type(x).__name__}")


def _matrix(x, name, rows=None, cols=None):
    """(rows, columns, row stride) of a bfloat16 matrix of the given shape with contiguous rows."""
    try:
        shape, dtype = x.shape, x.dtype
    except AttributeError:
        raise _no_tensor(x, name) from None
    if dtype is not _bf16:
        raise TypeError(f"{name} must be bfloat16, got {dtype}")
    if len(shape) != 2:
        raise TypeError(f"{name} must have 2 dimensions")
    r, c = shape
    ld, inner = x.stride()
    if inner != 1 and c > 1:
        raise TypeError(f"{name}: the last dimension must be contiguous")
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} must have shape ({'any' if rows is None else rows}, {'any' if cols is None else cols}), got ({r}, {c})")
    return r, c, ld if r > 1 and c else c or 1


def _columns(x, name):
    """The columns of a matrix that _kept() then looks at."""
    shape = getattr(x, "shape", ())
    if len(shape) != 2:
        raise TypeError(f"{name} must be a matrix")
    return shape[1]


def _code(dtype, name) -> int:
    """enum sgemm_type of an output's type (None: bfloat16)."""
    t = 1 if dtype is None else fp8._TYPES.get(dtype)
    if t is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")
    return t


def _act(activation) -> int:
    try:
        return ACTIVATIONS[activation]
    except (KeyError, TypeError):
        raise ValueError(f"unknown activation {activation!r}: None, 'relu', 'silu', 'gelu' or 'gelu_tanh'") from None


def _kept(k, name, rows, cols):
    """(structure, device number) of a matrix that was kept: bfloat16, or an Fp8Matrix of E4M3 codes in groups of (1, 128)."""
    if type(k) is Fp8Matrix:
        c = k._c()
        if k._shape != (rows, cols):
            raise ValueError(f"{name} must have shape ({rows}, {cols}), got {tuple(k._shape)}")
        if k._block != ROW or c.format != 0:
            raise ValueError(f"{name} must have E4M3 codes and groups of (1, 128)")
        return KeptStruct(c.data, c.ld, c.scale, c.lds), k._device
    ld = _matrix(k, name, rows, cols)[2]
    return KeptStruct(k.data_ptr(), ld, None, 1), k.get_device()


def _alloc(rows, cols, dtype, like, stream):
    """(tensor, row stride): uninitialised, its rows at multiples of 8 elements, as the kernels write them fastest."""
    ld = (cols + 7) & ~7
    return _empty((rows, cols), dtype, like, stream, None if ld == cols else ld), ld or 1


def _keep(how, rows, cols, like, stream):
    """(what a forward pass returns, its structure) for values that are kept."""
    if how == "fp8":
        m = _new_matrix(rows, cols, ROW, 0, like, stream)
        c = m._struct
        return m, KeptStruct(c.data, c.ld, c.scale, c.lds)
    t, ld = _alloc(rows, cols, _bf16, like, stream)
    return t, KeptStruct(t.data_ptr(), ld, None, 1)


def _check_keep(save):
    if save not in KEEP:
        raise ValueError(f"save must be None, 'bf16' or 'fp8', got {save!r}")


LinearOutput = namedtuple("LinearOutput", "y pre")
LinearGradients = namedtuple("LinearGradients", "dx dweight dbias")
GatedOutput = namedtuple("GatedOutput", "h gate up")
GatedGradients = namedtuple("GatedGradients", "dx dgate dup h")


def linear_bf16(x, weight, bias=None, activation=None, residual=None, *, save=None, out=None, out_dtype=None, stream=None) -> LinearOutput:
    """act(x weight^T + bias) + residual of a layer (sgemm_linear): x [tokens, inputs], weight [outputs, inputs], bias
    [outputs] and residual [tokens, outputs], all bfloat16; activation None, "relu", "silu", "gelu" or "gelu_tanh".

    Returns (y, pre): `y` in bfloat16 unless out_dtype or out says float32 (out may be a bfloat16 residual), `pre` the values
    before the activation where save is "bf16" or "fp8" (an Fp8Matrix), else None."""
    lib = _lib()
    tokens, inputs, ldx = _matrix(x, "x")
    outputs, _, ldw = _matrix(weight, "weight", None, inputs)
    act = _act(activation)
    _check_keep(save)
    if bias is not None:
        try:
            fp8._vector(bias, "bias", outputs, _bf16)
        except AttributeError:
            raise _no_tensor(bias, "bias") from None
    r_ptr, ldr = None, 0
    if residual is not None:
        ldr = _matrix(residual, "residual", tokens, outputs)[2]
        r_ptr = residual.data_ptr()
    if out is not None:
        try:
            rows, cols, ldy = _rows(out, "out")
        except AttributeError:
            raise _no_tensor(out, "out") from None
        if rows != tokens or cols != outputs:
            raise ValueError("out has the wrong shape")
        if out_dtype is not None and out.dtype is not out_dtype:
            raise TypeError(f"out is {out.dtype}, not {out_dtype}")
    t = _code(out_dtype if out is None else out.dtype, "out")
    handle = _on(stream, x.get_device(), weight, bias, residual, out)
    y = out
    if y is None:
        y, ldy = _alloc(tokens, outputs, out_dtype or _bf16, x, stream)
    pre = kept = None
    if save is not None:
        pre, kept = _keep(save, tokens, outputs, x, stream)
    st = lib.sgemm_linear(tokens, inputs, outputs, x.data_ptr(), ldx, weight.data_ptr(), ldw, None if bias is None else bias.data_ptr(), act,
                          r_ptr, ldr, kept, y.data_ptr(), ldy, t, handle)
    if st != 0:
        raise SgemmError(st, "sgemm_linear")
    return LinearOutput(y, pre)


def linear_bf16_backward(dy, x, weight, pre=None, activation=None, *, dx=True, dweight=True, dbias=False, dweight_dtype=None,
                         stream=None) -> LinearGradients:
    """The gradients of linear_bf16 from that of its output (sgemm_linear_backward): with d = dy * act'(pre), dx = d weight,
    dweight = d^T x and dbias the sum of d over the tokens (the residual's gradient is dy).

    pre: as the forward pass saved it, needed where there is an activation; x: bfloat16, or an Fp8Matrix with E4M3 codes and
    groups of (1, 128).  dx, dweight and dbias say which are wanted (None is returned for the others; x and weight may then be None
    where they are not needed).  dx is bfloat16, dweight bfloat16 unless dweight_dtype says float32, dbias float32."""
    lib = _lib()
    tokens, outputs, lddy = _matrix(dy, "dy")
    act = _act(activation)
    inputs, w_ptr, ldw, xs, x_dev, ks, k_dev = 0, None, 1, None, None, None, None
    if dx:
        _, inputs, ldw = _matrix(weight, "weight", outputs)
        w_ptr = weight.data_ptr()
    else:
        weight = None
    if dweight:
        if not dx:
            inputs = _columns(x, "x")
        xs, x_dev = _kept(x, "x", tokens, inputs)
    if act:
        if pre is None:
            raise ValueError("an activation's gradient needs pre")
        ks, k_dev = _kept(pre, "pre", tokens, outputs)
    t = _code(dweight_dtype, "dweight")
    handle = _on(stream, dy.get_device(), weight, x_dev, k_dev)
    gx = gw = gb = gx_ptr = gw_ptr = gb_ptr = None
    lddx = lddw = 1
    if dx:
        gx, lddx = _alloc(tokens, inputs, _bf16, dy, stream)
        gx_ptr = gx.data_ptr()
    if dweight:
        gw, lddw = _alloc(outputs, inputs, dweight_dtype or _bf16, dy, stream)
        gw_ptr = gw.data_ptr()
    if dbias:
        gb = _empty((outputs,), _f32, dy, stream)
        gb_ptr = gb.data_ptr()
    st = lib.sgemm_linear_backward(tokens, inputs, outputs, dy.data_ptr(), lddy, xs, w_ptr, ldw, act, ks, gx_ptr, lddx, gw_ptr, lddw, t, gb_ptr, handle)
    if st != 0:
        raise SgemmError(st, "sgemm_linear_backward")
    return LinearGradients(gx, gw, gb)


def gated_bf16(x, gate, up, activation="silu", *, save=None, out=None, stream=None) -> GatedOutput:
    """act(x gate^T) * (x up^T), the first half of a gated feed-forward block in one kernel (sgemm_gated): x [tokens,
    inputs], gate and up [outputs, inputs], bfloat16.

    Returns (h, gate, up): `h` in bfloat16, and both products where save is "bf16" or "fp8" (an Fp8Matrix each), else None."""
    lib = _lib()
    tokens, inputs, ldx = _matrix(x, "x")
    outputs, _, ldg = _matrix(gate, "gate", None, inputs)
    ldu = _matrix(up, "up", outputs, inputs)[2]
    act = _act(activation)
    _check_keep(save)
    if out is not None:
        ldh = _matrix(out, "out", tokens, outputs)[2]
    handle = _on(stream, x.get_device(), gate, up, out)
    h = out
    if h is None:
        h, ldh = _alloc(tokens, outputs, _bf16, x, stream)
    a = b = ka = kb = None
    if save is not None:
        a, ka = _keep(save, tokens, outputs, x, stream)
        b, kb = _keep(save, tokens, outputs, x, stream)
    st = lib.sgemm_gated(tokens, inputs, outputs, x.data_ptr(), ldx, gate.data_ptr(), ldg, up.data_ptr(), ldu, act, ka, kb, h.data_ptr(), ldh,
                         handle)
    if st != 0:
        raise SgemmError(st, "sgemm_gated")
    return GatedOutput(h, a, b)


def gated_bf16_backward(dh, x, gate, up, gate_pre, up_pre, activation="silu", *, dx=True, dweights=True, h=False, dweight_dtype=None,
                        stream=None) -> GatedGradients:
    """The gradients of gated_bf16 from that of h (sgemm_gated_backward): with a and b the two products as the forward pass
    saved them, da = dh * b * act'(a) and db = dh * act(a), dx = da gate + db up, dgate = da^T x, dup = db^T x.

    h=True: act(a) * b too, in bfloat16, which the weight gradient of the layer behind needs.  x: bfloat16, or an Fp8Matrix
    with E4M3 codes and groups of (1, 128).  dx and dweights say which are wanted (None is returned for the others)."""
    lib = _lib()
    tokens, outputs, lddh = _matrix(dh, "dh")
    act = _act(activation)
    inputs, ldg, ldu, g_ptr, u_ptr, xs, x_dev = 0, 1, 1, None, None, None, None
    if dx:
        _, inputs, ldg = _matrix(gate, "gate", outputs)
        _, _, ldu = _matrix(up, "up", outputs, inputs)
        g_ptr, u_ptr = gate.data_ptr(), up.data_ptr()
    else:
        gate = up = None
    if dweights:
        if not dx:
            inputs = _columns(x, "x")
        xs, x_dev = _kept(x, "x", tokens, inputs)
    ka, a_dev = _kept(gate_pre, "gate_pre", tokens, outputs)
    kb, b_dev = _kept(up_pre, "up_pre", tokens, outputs)
    if (type(gate_pre) is Fp8Matrix) != (type(up_pre) is Fp8Matrix):
        raise TypeError("gate_pre and up_pre must be kept alike")
    t = _code(dweight_dtype, "dgate and dup")
    handle = _on(stream, dh.get_device(), gate, up, x_dev, a_dev, b_dev)
    gx = dg = du = ho = gx_ptr = dg_ptr = du_ptr = ho_ptr = None
    lddx = ldw = ldh = 1
    if dx:
        gx, lddx = _alloc(tokens, inputs, _bf16, dh, stream)
        gx_ptr = gx.data_ptr()
    if dweights:
        dtype = dweight_dtype or _bf16
        dg, ldw = _alloc(outputs, inputs, dtype, dh, stream)
        du, _ = _alloc(outputs, inputs, dtype, dh, stream)
        dg_ptr, du_ptr = dg.data_ptr(), du.data_ptr()
    if h:
        ho, ldh = _alloc(tokens, outputs, _bf16, dh, stream)
        ho_ptr = ho.data_ptr()
    st = lib.sgemm_gated_backward(tokens, inputs, outputs, dh.data_ptr(), lddh, xs, g_ptr, ldg, u_ptr, ldu, act, ka, kb, gx_ptr, lddx, dg_ptr, ldw,
                                  du_ptr, ldw, t, ho_ptr, ldh, handle)
    if st != 0:
        raise SgemmError(st, "sgemm_gated_backward")
    return GatedGradients(gx, dg, du, ho)


def sgemm_linear_plan(rows, cols, K, gated=False, kept8=False, sm_count=0) -> dict:
    """The launch this part makes for a product of rows x cols over K of aligned matrices.  Raises on invalid arguments."""
    plan = PlanStruct()
    st = _lib().sgemm_linear_plan(rows, cols, K, int(gated), int(kept8), sm_count, ctypes.byref(plan))
    if st != 0:
        raise SgemmError(st, "sgemm_linear_plan")
    out = {name: getattr(plan, name) for name, _ in PlanStruct._fields_}
    out["variant_name"] = VARIANTS.get(out["variant"], str(out["variant"]))
    return out


def sgemm_linear_set_override(variant="AUTO", tile_n=0, split=0) -> None:
    """Forces this part's kernel ("LINEAR_PAIR", "LINEAR_SHORT"; "AUTO" restores the planner's choice), tile and K split."""
    names = {v: k for k, v in VARIANTS.items()}
    st = _lib().sgemm_linear_set_override(names[variant], tile_n, split)
    if st != 0:
        raise SgemmError(st, "sgemm_linear_set_override")
