"""The 8-bit operators of libsgemm (C ABI in include/sgemm_fp8.h): argument marshalling only.

An ``Fp8Matrix`` is a 2-D tensor of 8-bit codes with the scales of its groups of
1x128, 128x1 or 128x128 elements.  ``quantize_fp8`` makes one from an FP32 or
BF16 matrix, ``rmsnorm_fp8`` makes one from a layer's input, ``matmul_fp8``
multiplies two, ``moe_fp8`` runs a mixture-of-experts layer on one.  Outputs
that a call allocates belong to the stream it runs on; rows of codes start at
multiples of 16 elements and rows of the norm's outputs at multiples of 8.  A
call's tensors are on one device, which is the current one (ValueError otherwise).
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

from . import PlanStruct, SgemmError, _ch, _stream, load

FORMATS = {"e4m3": 0, "e5m2": 1}
VARIANTS = {0: "AUTO", 1: "NONE", 2: "SCALE", 32: "FP8_PAIR", 33: "FP8_SHORT"}
ROW, COL, BLOCK = (1, 128), (128, 1), (128, 128)
GROUPS = (ROW, COL, BLOCK)


class MatrixStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("scale", ctypes.c_void_p), ("lds", ctypes.c_int64),
                ("format", ctypes.c_int), ("block_rows", ctypes.c_int), ("block_cols", ctypes.c_int)]


class ExpertsStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("stride", ctypes.c_int64), ("scale", ctypes.c_void_p),
                ("lds", ctypes.c_int64), ("stride_scale", ctypes.c_int64)]


_functions = None  # the compiled library, once its signatures are set
_T = None          # torch, imported with the first call
_CODES = {}        # torch dtype -> enum sgemm_fp8_format
_TYPES = {}        # torch dtype -> enum sgemm_type
_raw_stream = None
_current_device = None


def _declare(lib):
    """C signatures of this file's entry points."""
    i64, f32, vp, ci = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
    mp, ep, ch = ctypes.POINTER(MatrixStruct), ctypes.POINTER(ExpertsStruct), ctypes.c_char
    for name, args in {
        "sgemm_fp8": [ch, ch, i64, i64, i64, f32, mp, mp, f32, vp, i64, vp, i64, ci, vp],
        "sgemm_fp8_plan": [ch, ch, i64, i64, i64, f32, mp, mp, f32, vp, i64, vp, i64, ci, ci, ctypes.POINTER(PlanStruct)],
        "sgemm_fp8_set_override": [ci, ci, ci],
        "sgemm_fp8_moe": [i64, i64, i64, i64, ci, mp, vp, i64, ci, ep, ep, ep, vp, i64, ci, vp],
        "sgemm_fp8_quantize": [i64, i64, vp, ci, i64, ci, ci, ci, vp, i64, vp, i64, vp],
        "sgemm_fp8_rmsnorm": [i64, i64, ci, vp, i64, vp, i64, vp, f32, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp],
        "sgemm_fp8_rmsnorm_backward": [i64, i64, ci, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp],
    }.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = ci, args
    return lib


def _lib():
    """The compiled library with the C signatures of this file's entry points."""
    global _functions, _T, _raw_stream, _current_device
    if _functions is None:
        import torch
        lib = _declare(load())
        _CODES.update({torch.float8_e4m3fn: 0, torch.float8_e5m2: 1})
        _TYPES.update({torch.float32: 0, torch.bfloat16: 1})
        # the handle alone: torch.cuda.current_stream() builds an object, which costs as much as a launch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _T, _functions = torch, lib
    return _functions


def _not_cuda():
    return TypeError("operands must be CUDA tensors")


def _on(stream, device, *others):
    """The stream handle a call on the current device runs on.  device: that of the first operand, others: further tensors
    or device numbers (None: not given); the library launches on the current device, so another one is refused."""
    for t in others:
        if t is not None:
            d = t if type(t) is int else t.get_device()
            if d != device:
                raise ValueError(f"operands on cuda:{device} and cuda:{d}: all must be on one device") if d >= 0 else _not_cuda()
    if device < 0:
        raise _not_cuda()
    if device != _current_device():
        raise ValueError(f"operands are on cuda:{device}, the current device is cuda:{_current_device()}")
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    if getattr(getattr(stream, "device", None), "index", device) != device:
        raise ValueError(f"operands are on cuda:{device}, the stream on {stream.device}")
    return _stream(stream)


def _type(x, name) -> int:
    t = _TYPES.get(x.dtype)
    if t is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {x.dtype}")
    return t


def _rows(x, name):
    """(rows, columns, row stride) of a 2-D tensor with contiguous rows (a single row has no stride of its own)."""
    shape = x.shape
    if len(shape) != 2:
        raise TypeError(f"{name} must have 2 dimensions")
    rows, cols = shape
    ld, inner = x.stride()
    if inner != 1 and cols > 1:
        raise TypeError(f"{name}: the last dimension must be contiguous")
    if rows <= 1 or cols == 0:
        ld = cols or 1
    return rows, cols, ld


def _empty(shape, dtype, like, stream, ld=None):
    """Uninitialised memory that belongs to the stream the call runs on; ld: the row stride where it is not the width."""
    if stream is None:
        if ld is not None:
            return _T.empty_strided(shape, (ld, 1), dtype=dtype, device=like.device)
        return _T.empty(shape, dtype=dtype, device=like.device)
    if not hasattr(stream, "cuda_stream"):
        stream = _T.cuda.ExternalStream(int(stream), device=like.device) if stream else _T.cuda.default_stream(like.device)
    with _T.cuda.stream(stream):
        return _empty(shape, dtype, like, None, ld)


def _empty_rows(rows, cols, like, stream):
    """(tensor, row stride): an uninitialised rows x cols tensor of like's type whose rows start at multiples of 16
    bytes, as the kernels write them fastest."""
    ld = (cols + 7) // 8 * 8
    return _empty((rows, cols), like.dtype, like, stream, None if ld == cols else ld), ld or 1


class Fp8Matrix:
    """A stored matrix of 8-bit codes: ``data`` (2-D, float8_e4m3fn or float8_e5m2, rows contiguous), ``scale``
    (float32, one per group, rows contiguous) and ``block``, the elements (rows, columns) of a group.

    Element (r, c) is ``data[r, c] * scale[r // block[0], c // block[1]]``.  The attributes are fixed; the tensors' values
    may change between calls, and so may their memory (``tensor.data = other``) as long as the shapes stay."""

    __slots__ = ("_data", "_scale", "_block", "_shape", "_struct", "_at", "_device")

    data = property(lambda self: self._data)
    scale = property(lambda self: self._scale)
    block = property(lambda self: self._block)
    shape = property(lambda self: self._shape)

    def __init__(self, data, scale, block=ROW):
        _lib()
        fmt = _CODES.get(data.dtype)
        if fmt is None:
            raise TypeError(f"data must be float8_e4m3fn or float8_e5m2, got {data.dtype}")
        if scale.dtype is not _T.float32:
            raise TypeError(f"scale must be float32, got {scale.dtype}")
        rows, cols, ld = _rows(data, "data")
        srows, scols, lds = _rows(scale, "scale")
        device = data.get_device()
        if device < 0:
            raise _not_cuda()
        if scale.get_device() != device:
            raise ValueError(f"data is on cuda:{device}, scale on cuda:{scale.get_device()}")
        br, bc = block
        if (br, bc) not in GROUPS:
            raise ValueError("block must be (1, 128), (128, 1) or (128, 128)")
        if srows != -(-rows // br) or scols != -(-cols // bc):
            raise ValueError(f"scale must have shape {(-(-rows // br), -(-cols // bc))}, got {(srows, scols)}")
        self._data, self._scale, self._block, self._shape = data, scale, (br, bc), data.shape
        self._at, self._device = (data.data_ptr(), scale.data_ptr()), device
        self._struct = MatrixStruct(self._at[0], ld, self._at[1], lds, fmt, br, bc)

    def _c(self):
        """The C structure; made again where a tensor's memory is no longer the one it was made for."""
        if (self._data.data_ptr(), self._scale.data_ptr()) != self._at:
            if self._data.shape != self._shape:
                raise ValueError(f"data had shape {tuple(self._shape)}, has {tuple(self._data.shape)}")
            self.__init__(self._data, self._scale, self._block)
        return self._struct


def _new_matrix(rows, cols, block, fmt, like, stream):
    """An Fp8Matrix of uninitialised codes and scales; rows start at multiples of 16 bytes."""
    dtype = _T.float8_e5m2 if fmt else _T.float8_e4m3fn
    ld = (cols + 15) // 16 * 16
    data = _empty((rows, cols), dtype, like, stream, None if ld == cols else ld)
    br, bc = block
    scols = -(-cols // bc)
    m = Fp8Matrix.__new__(Fp8Matrix)
    m._scale = scale = _empty((-(-rows // br), scols), _T.float32, like, stream)
    m._data, m._block, m._shape = data, block, data.shape
    m._at = at = (data.data_ptr(), scale.data_ptr())
    m._device = data.get_device()
    m._struct = MatrixStruct(at[0], ld or 1, at[1], scols or 1, fmt, br, bc)
    return m


def quantize_fp8(x, block=ROW, format="e4m3", stream=None) -> Fp8Matrix:
    """Codes and scales of a 2-D float32 or bfloat16 tensor in groups of `block` elements: (1, 128), (128, 1) or
    (128, 128).  For each group the scale is max(amax / top, 2**-126) and the code of x is x * (1 / scale) rounded
    to nearest even (sgemm_fp8_quantize).  Rows of the codes start at multiples of 16 elements: where the width is not one,
    ``data`` is not contiguous."""
    lib = _lib()
    rows, cols, ldx = _rows(x, "x")
    fmt = FORMATS.get(format)
    if fmt is None:
        raise ValueError(f"unknown 8-bit format {format!r}")
    t = _type(x, "x")
    block = tuple(block)
    if block not in GROUPS:
        raise ValueError("block must be (1, 128), (128, 1) or (128, 128)")
    handle = _on(stream, x.get_device())
    m = _new_matrix(rows, cols, block, fmt, x, stream)
    c = m._struct
    st = lib.sgemm_fp8_quantize(rows, cols, x.data_ptr(), t, ldx, fmt, block[0], block[1], c.data, c.ld, c.scale, c.lds, handle)
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_quantize")
    return m


_OPS = {"N": (False, b"N"), "n": (False, b"N"), "T": (True, b"T"), "t": (True, b"T"), "C": (True, b"T"), "c": (True, b"T")}


def matmul_fp8(A: Fp8Matrix, B: Fp8Matrix, C=None, transA="N", transB="N", alpha=1.0, beta=0.0, *, out=None, out_dtype=None,
               stream=None):
    """alpha * op(A) op(B) + beta * C on 8-bit matrices (sgemm_fp8), float32 or bfloat16.

    A and B are the stored matrices; both must have groups of 128 along the summed dimension.  The result goes to `out`, else
    to C in place, else to a new tensor of `out_dtype` (float32 unless given)."""
    lib = _lib()
    a, b = A._c(), B._c()
    try:
        (ta, opa), (tb, opb) = _OPS[transA], _OPS[transB]
    except KeyError:
        raise ValueError(f"unknown operation {transA!r} or {transB!r}: N or T") from None
    M, K = A._shape
    if ta:
        M, K = K, M
    kb, N = B._shape
    if tb:
        kb, N = N, kb
    if kb != K:
        raise ValueError("inner dimensions of op(A) and op(B) differ")
    c_ptr, ldc = None, N or 1
    d = out
    if C is not None:
        rows, cols, ldc = _rows(C, "C")
        if rows != M or cols != N:
            raise ValueError("C has the wrong shape")
        if d is None:
            d = C
        elif d.dtype is not C.dtype:
            raise TypeError(f"C is {C.dtype} and out is {d.dtype}")
        c_ptr = C.data_ptr()
    elif beta != 0.0:
        raise ValueError("beta != 0 needs C")
    handle = _on(stream, A._device, B._device, C, d)
    if d is None:
        d = _empty((M, N), out_dtype or _T.float32, A._data, stream)
    elif out_dtype is not None and d.dtype is not out_dtype:
        raise TypeError(f"out is {d.dtype}, not {out_dtype}")
    t = _type(d, "out")
    rows, cols, ldd = _rows(d, "out")
    if rows != M or cols != N:
        raise ValueError("out has the wrong shape")
    st = lib.sgemm_fp8(opa, opb, M, N, K, alpha, a, b, beta, c_ptr, ldc, d.data_ptr(), ldd, t, handle)
    if st != 0:
        raise SgemmError(st, "sgemm_fp8")
    return d


def sgemm_fp8_plan(transA, transB, M, N, K, alpha, A, B, beta, C, ldc, D, ldd, type, sm_count=0) -> dict:
    """The launch sgemm_fp8() would make; A and B are MatrixStructs.  Raises on invalid arguments."""
    plan = PlanStruct()
    st = _lib().sgemm_fp8_plan(_ch(transA), _ch(transB), M, N, K, alpha, A, B, beta, C, ldc, D, ldd, type, sm_count,
                               ctypes.byref(plan))
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_plan")
    out = {name: getattr(plan, name) for name, _ in PlanStruct._fields_}
    out["variant_name"] = VARIANTS.get(out["variant"], str(out["variant"]))
    return out


def sgemm_fp8_set_override(variant="AUTO", tile_n=0, split=0) -> None:
    """Forces sgemm_fp8()'s kernel ("FP8_PAIR", "FP8_SHORT"; "AUTO" restores the planner's choice), tile and K split."""
    names = {v: k for k, v in VARIANTS.items()}
    st = _lib().sgemm_fp8_set_override(names[variant], tile_n, split)
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_set_override")


NormOutput = namedtuple("NormOutput", "q h y rstd")
_NO_MATRIX = MatrixStruct()


def _vector(x, name, n, dtype):
    if x.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if x.shape != (n,):
        raise ValueError(f"{name} must have shape ({n},), got {tuple(x.shape)}")
    if n > 1 and x.stride(0) != 1:
        raise TypeError(f"{name} must be contiguous")


def rmsnorm_fp8(x, weight, eps=1e-6, residual=None, *, codes=True, y=False, stream=None) -> NormOutput:
    """h = x + residual, then y = h * rstd * weight with rstd = (mean(h**2) + eps)**-0.5 along each row
    (sgemm_fp8_rmsnorm).

    Returns (q, h, y, rstd): `q` the E4M3 codes and scales of y in groups of (1, 128) (None with codes=False), `h` the sum
    (x itself without a residual), `y` in x's type when y=True (else None), `rstd` float32 of one value per row.  Where the
    width is no multiple of 8, `h` and `y` are not contiguous (their rows start at multiples of 8 elements)."""
    lib = _lib()
    t = _type(x, "x")
    rows, cols, ldx = _rows(x, "x")
    dtype = x.dtype
    _vector(weight, "weight", cols, dtype)
    handle = _on(stream, x.get_device(), weight, residual)
    h, r_ptr, ldr, h_ptr, ldh = x, None, 0, None, cols or 1
    if residual is not None:
        rrows, rcols, ldr = _rows(residual, "residual")
        if rrows != rows or rcols != cols or residual.dtype is not dtype:
            raise ValueError("residual must have x's shape and type")
        h, ldh = _empty_rows(rows, cols, x, stream)
        r_ptr, h_ptr = residual.data_ptr(), h.data_ptr()
    out, ldy = _empty_rows(rows, cols, x, stream) if y else (None, cols or 1)
    rstd = _empty((rows,), _T.float32, x, stream)
    q = _new_matrix(rows, cols, ROW, 0, x, stream) if codes else None
    c = q._struct if codes else _NO_MATRIX
    st = lib.sgemm_fp8_rmsnorm(rows, cols, t, x.data_ptr(), ldx, r_ptr, ldr, weight.data_ptr(), eps, h_ptr, ldh,
                               out.data_ptr() if y else None, ldy, c.data, c.ld, c.scale, c.lds, rstd.data_ptr(), handle)
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_rmsnorm")
    return NormOutput(q, h, out, rstd)


def rmsnorm_fp8_backward(dy, h, weight, rstd, dh=None, *, stream=None):
    """(dx, dweight) of rmsnorm_fp8: `dy` the gradient of y, `h` and `rstd` as the forward pass returned them, `dh` the
    gradient that reaches h past the norm.  dx is the gradient of x and of the residual, not contiguous where the width is no
    multiple of 8; dweight is float32."""
    lib = _lib()
    t = _type(dy, "dy")
    rows, cols, lddy = _rows(dy, "dy")
    dtype = dy.dtype
    _vector(weight, "weight", cols, dtype)
    _vector(rstd, "rstd", rows, _T.float32)
    hrows, hcols, ldh = _rows(h, "h")
    if hrows != rows or hcols != cols or h.dtype is not dtype:
        raise ValueError("h must have dy's shape and type")
    dh_ptr, lddh = None, 0
    if dh is not None:
        drows, dcols, lddh = _rows(dh, "dh")
        if drows != rows or dcols != cols or dh.dtype is not dtype:
            raise ValueError("dh must have dy's shape and type")
        dh_ptr = dh.data_ptr()
    handle = _on(stream, dy.get_device(), h, weight, rstd, dh)
    dx, lddx = _empty_rows(rows, cols, dy, stream)
    dw = _empty((cols,), _T.float32, dy, stream)
    st = lib.sgemm_fp8_rmsnorm_backward(rows, cols, t, dy.data_ptr(), lddy, h.data_ptr(), ldh, weight.data_ptr(), rstd.data_ptr(),
                                        dh_ptr, lddh, dx.data_ptr(), lddx, dw.data_ptr(), handle)
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_rmsnorm_backward")
    return dx, dw


def _stack(x, name, shape, dtype):
    """(stride between matrices, row stride) of a 3-D tensor of `shape` with contiguous rows."""
    if len(x.shape) != 3:
        raise TypeError(f"{name} must have 3 dimensions")
    if x.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(x.shape)}")
    stride, ld, inner = x.stride()
    if inner != 1 and shape[2] > 1:
        raise TypeError(f"{name}: the last dimension must be contiguous")
    return stride, ld


def _experts(w, name, experts, rows, cols) -> ExpertsStruct:
    data, scale = w
    stride, ld = _stack(data, name, (experts, rows, cols), _T.float8_e4m3fn)
    sstride, lds = _stack(scale, name + " scales", (experts, -(-rows // 128), -(-cols // 128)), _T.float32)
    return ExpertsStruct(data.data_ptr(), ld, stride, scale.data_ptr(), lds or 1, sstride)


def moe_fp8(x: Fp8Matrix, logits, top_k, gate, up, down, *, renormalize=True, out=None, out_dtype=None, stream=None):
    """A mixture-of-experts layer for a few tokens (sgemm_fp8_moe): for each row t of x the sum over the `top_k` experts with
    the largest logits (ties: lowest index) of their softmax weight times down_e (silu(gate_e x_t) * (up_e x_t)).

    x: E4M3 with groups of (1, 128), at most 64 rows; logits: float32 [tokens, experts]; gate and up: (codes [experts, inner,
    hidden], scales [experts, inner / 128, hidden / 128]) with groups of 128 x 128, down: [experts, hidden, inner].  The
    weights are divided by their sum over the chosen experts with renormalize=True.  Returns bfloat16 unless out_dtype or
    out says otherwise."""
    lib = _lib()
    xs = x._c()
    tokens, hidden = x._shape
    experts, inner = gate[0].shape[:2]
    lrows, lcols, ldl = _rows(logits, "logits")
    if logits.dtype is not _T.float32:
        raise TypeError("logits must be float32")
    if lrows != tokens or lcols != experts:
        raise ValueError("logits must have one value per token and expert")
    g = _experts(gate, "gate", experts, inner, hidden)
    u = _experts(up, "up", experts, inner, hidden)
    d = _experts(down, "down", experts, hidden, inner)
    handle = _on(stream, x._device, logits, *gate, *up, *down, out)
    y = out if out is not None else _empty((tokens, hidden), out_dtype or _T.bfloat16, x._data, stream)
    yrows, ycols, ldy = _rows(y, "out")
    if yrows != tokens or ycols != hidden:
        raise ValueError("out has the wrong shape")
    t = _type(y, "out")
    if out_dtype is not None and y.dtype is not out_dtype:
        raise TypeError(f"out is {y.dtype}, not {out_dtype}")
    st = lib.sgemm_fp8_moe(tokens, hidden, inner, experts, top_k, xs, logits.data_ptr(), ldl, 1 if renormalize else 0, g, u, d,
                           y.data_ptr(), ldy, t, handle)
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_moe")
    return y
