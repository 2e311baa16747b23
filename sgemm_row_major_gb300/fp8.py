"""The 8-bit operators of libsgemm (C ABI in include/sgemm_fp8.h): argument marshalling only.

An ``Fp8Matrix`` is a 2-D tensor of 8-bit codes with the scales of its groups of
1x128, 128x1 or 128x128 elements.  ``quantize_fp8`` makes one from an FP32 or
BF16 matrix, ``rmsnorm_fp8`` makes one from a layer's input, ``matmul_fp8``
multiplies two, ``moe_fp8`` runs a mixture-of-experts layer on one.  Outputs
that a call allocates belong to the stream it runs on.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

from . import PlanStruct, SgemmError, _ch, _stream, load

FORMATS = {"e4m3": 0, "e5m2": 1}
VARIANTS = {0: "AUTO", 1: "NONE", 2: "SCALE", 32: "FP8_PAIR", 33: "FP8_SHORT"}
ROW, COL, BLOCK = (1, 128), (128, 1), (128, 128)


class MatrixStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("scale", ctypes.c_void_p), ("lds", ctypes.c_int64),
                ("format", ctypes.c_int), ("block_rows", ctypes.c_int), ("block_cols", ctypes.c_int)]


class ExpertsStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("stride", ctypes.c_int64), ("scale", ctypes.c_void_p),
                ("lds", ctypes.c_int64), ("stride_scale", ctypes.c_int64)]


_functions = None


def _lib():
    """The compiled library with the C signatures of this file's entry points."""
    global _functions
    if _functions is None:
        lib = load()
        i64, f32, vp, ci = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
        mp, ep, ch = ctypes.POINTER(MatrixStruct), ctypes.POINTER(ExpertsStruct), ctypes.c_char
        lib.sgemm_fp8_plan.restype = ci
        lib.sgemm_fp8_plan.argtypes = [ch, ch, i64, i64, i64, f32, mp, mp, f32, vp, i64, vp, i64, ci, ci, ctypes.POINTER(PlanStruct)]
        for name, args in {
            "sgemm_fp8": [ch, ch, i64, i64, i64, f32, mp, mp, f32, vp, i64, vp, i64, ci, vp],
            "sgemm_fp8_set_override": [ci, ci, ci],
            "sgemm_fp8_moe": [i64, i64, i64, i64, ci, mp, vp, i64, ci, ep, ep, ep, vp, i64, ci, vp],
            "sgemm_fp8_quantize": [i64, i64, vp, ci, i64, ci, ci, ci, vp, i64, vp, i64, vp],
            "sgemm_fp8_rmsnorm": [i64, i64, ci, vp, i64, vp, i64, vp, f32, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp],
            "sgemm_fp8_rmsnorm_backward": [i64, i64, ci, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp],
        }.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = ci, args
        _functions = lib
    return _functions


def _type(dtype) -> int:
    import torch
    if dtype == torch.float32:
        return 0
    if dtype == torch.bfloat16:
        return 1
    raise TypeError(f"expected a float32 or bfloat16 tensor, got {dtype}")


def _check(x, name, dims=2, dtype=None):
    if not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if x.dim() != dims:
        raise TypeError(f"{name} must have {dims} dimension(s)")
    if dtype is not None and x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if x.shape[-1] > 1 and x.stride(-1) != 1:
        raise TypeError(f"{name}: the last dimension must be contiguous")
    return x


def _ld(x) -> int:
    """Row stride of a 2-D tensor (a single row has none of its own)."""
    return max(x.stride(0) if x.shape[0] > 1 else x.shape[1], 1)


def _empty(shape, dtype, like, stream):
    """Uninitialised memory that belongs to the stream the call runs on."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device) if stream else torch.cuda.default_stream(like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _code_dtypes():
    import torch
    return {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}


class Fp8Matrix:
    """A stored matrix of 8-bit codes: ``data`` (2-D, float8_e4m3fn or float8_e5m2, rows contiguous), ``scale``
    (float32, one per group, rows contiguous) and ``block``, the elements (rows, columns) of a group.

    Element (r, c) is ``data[r, c] * scale[r // block[0], c // block[1]]``."""

    __slots__ = ("data", "scale", "block", "_struct")

    def __init__(self, data, scale, block=ROW):
        import torch
        fmt = 0 if data.dtype == torch.float8_e4m3fn else 1 if data.dtype == torch.float8_e5m2 else None
        if fmt is None:
            raise TypeError(f"data must be float8_e4m3fn or float8_e5m2, got {data.dtype}")
        _check(data, "data")
        _check(scale, "scale", dtype=torch.float32)
        br, bc = block
        if (br, bc) not in (ROW, COL, BLOCK):
            raise ValueError("block must be (1, 128), (128, 1) or (128, 128)")
        rows, cols = data.shape
        if tuple(scale.shape) != (-(-rows // br), -(-cols // bc)):
            raise ValueError(f"scale must have shape {(-(-rows // br), -(-cols // bc))}, got {tuple(scale.shape)}")
        self.data, self.scale, self.block = data, scale, (br, bc)
        self._struct = MatrixStruct(data.data_ptr(), _ld(data), scale.data_ptr(), _ld(scale), fmt, br, bc)

    @property
    def shape(self):
        return self.data.shape


def _new_matrix(rows, cols, block, fmt, like, stream):
    """An Fp8Matrix of uninitialised codes and scales; rows start at multiples of 16 bytes."""
    import torch
    dtype = torch.float8_e5m2 if fmt else torch.float8_e4m3fn
    ld = (cols + 15) // 16 * 16
    data = _empty((rows, ld), dtype, like, stream)
    if ld != cols:
        data = data[:, :cols]
    return Fp8Matrix(data, _empty((-(-rows // block[0]), -(-cols // block[1])), torch.float32, like, stream), block)


def quantize_fp8(x, block=ROW, format="e4m3", stream=None) -> Fp8Matrix:
    """Codes and scales of a 2-D float32 or bfloat16 tensor in groups of `block` elements: (1, 128), (128, 1) or
    (128, 128).  For each group the scale is max(amax / top, 2**-126) and the code of x is x * (1 / scale) rounded
    to nearest even (sgemm_fp8_quantize)."""
    _check(x, "x")
    if format not in FORMATS:
        raise ValueError(f"unknown 8-bit format {format!r}")
    t = _type(x.dtype)
    if tuple(block) not in (ROW, COL, BLOCK):
        raise ValueError("block must be (1, 128), (128, 1) or (128, 128)")
    rows, cols = x.shape
    m = _new_matrix(rows, cols, block, FORMATS[format], x, stream)
    c = m._struct
    st = _lib().sgemm_fp8_quantize(rows, cols, x.data_ptr(), t, _ld(x), c.format, c.block_rows, c.block_cols, c.data, c.ld,
                                   c.scale, c.lds, _stream(stream))
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_quantize")
    return m


def _is_t(op) -> bool:
    op = op.decode() if isinstance(op, bytes) else str(op)
    if op[:1].upper() not in ("N", "T", "C"):
        raise ValueError(f"unknown operation {op!r}: N or T")
    return op[:1].upper() != "N"


def matmul_fp8(A: Fp8Matrix, B: Fp8Matrix, C=None, transA="N", transB="N", alpha=1.0, beta=0.0, *, out=None, out_dtype=None,
               stream=None):
    """alpha * op(A) op(B) + beta * C on 8-bit matrices (sgemm_fp8), float32 or bfloat16.

    A and B are the stored matrices; both must have groups of 128 along the summed dimension.  The result goes to `out`, else
    to C in place, else to a new tensor of `out_dtype` (float32 unless given)."""
    import torch
    ta, tb = _is_t(transA), _is_t(transB)
    M, K = A.data.shape[::-1] if ta else A.data.shape
    N, kb = B.data.shape if tb else B.data.shape[::-1]
    if kb != K:
        raise ValueError("inner dimensions of op(A) and op(B) differ")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        d = out if out is not None else _empty((M, N), out_dtype or torch.float32, A.data, stream)
        c_ptr, ldc = None, max(N, 1)
    else:
        d = out if out is not None else C
        _check(C, "C", 2, d.dtype)
        if tuple(C.shape) != (M, N):
            raise ValueError("C has the wrong shape")
        c_ptr, ldc = C.data_ptr(), _ld(C)
    t = _type(_check(d, "out").dtype)
    if tuple(d.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    if out_dtype is not None and d.dtype != out_dtype:
        raise TypeError(f"out is {d.dtype}, not {out_dtype}")
    st = _lib().sgemm_fp8(b"T" if ta else b"N", b"T" if tb else b"N", M, N, K, alpha, A._struct, B._struct, beta, c_ptr, ldc,
                          d.data_ptr(), _ld(d), t, _stream(stream))
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


def rmsnorm_fp8(x, weight, eps=1e-6, residual=None, *, codes=True, y=False, stream=None) -> NormOutput:
    """h = x + residual, then y = h * rstd * weight with rstd = (mean(h**2) + eps)**-0.5 along each row
    (sgemm_fp8_rmsnorm).

    Returns (q, h, y, rstd): `q` the E4M3 codes and scales of y in groups of (1, 128) (None with codes=False), `h` the sum
    (x itself without a residual), `y` in x's type when y=True (else None), `rstd` float32 of one value per row."""
    import torch
    t = _type(_check(x, "x").dtype)
    rows, cols = x.shape
    _check(weight, "weight", 1, x.dtype)
    if weight.shape[0] != cols:
        raise ValueError("weight must have one value per column of x")
    h, r_ptr, ldr, h_ptr, ldh = x, None, 0, None, 0
    if residual is not None:
        _check(residual, "residual", 2, x.dtype)
        if residual.shape != x.shape:
            raise ValueError("residual must have x's shape")
        h = _empty((rows, cols), x.dtype, x, stream)
        r_ptr, ldr, h_ptr, ldh = residual.data_ptr(), _ld(residual), h.data_ptr(), max(cols, 1)
    out = _empty((rows, cols), x.dtype, x, stream) if y else None
    rstd = _empty((rows,), torch.float32, x, stream)
    q = _new_matrix(rows, cols, ROW, 0, x, stream) if codes else None
    c = q._struct if codes else MatrixStruct()
    st = _lib().sgemm_fp8_rmsnorm(rows, cols, t, x.data_ptr(), _ld(x), r_ptr, ldr, weight.data_ptr(), eps, h_ptr, ldh,
                                  out.data_ptr() if y else None, max(cols, 1), c.data, c.ld, c.scale, c.lds, rstd.data_ptr(),
                                  _stream(stream))
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_rmsnorm")
    return NormOutput(q, h, out, rstd)


def rmsnorm_fp8_backward(dy, h, weight, rstd, dh=None, *, stream=None):
    """(dx, dweight) of rmsnorm_fp8: `dy` the gradient of y, `h` and `rstd` as the forward pass returned them, `dh` the
    gradient that reaches h past the norm.  dx is the gradient of x and of the residual; dweight is float32."""
    import torch
    t = _type(_check(dy, "dy").dtype)
    rows, cols = dy.shape
    _check(h, "h", 2, dy.dtype)
    _check(weight, "weight", 1, dy.dtype)
    _check(rstd, "rstd", 1, torch.float32)
    if h.shape != dy.shape or weight.shape[0] != cols or rstd.shape[0] != rows:
        raise ValueError("dy, h, weight and rstd do not belong together")
    if dh is not None:
        _check(dh, "dh", 2, dy.dtype)
        if dh.shape != dy.shape:
            raise ValueError("dh must have dy's shape")
    dx = _empty((rows, cols), dy.dtype, dy, stream)
    dw = _empty((cols,), torch.float32, dy, stream)
    st = _lib().sgemm_fp8_rmsnorm_backward(rows, cols, t, dy.data_ptr(), _ld(dy), h.data_ptr(), _ld(h), weight.data_ptr(),
                                           rstd.data_ptr(), None if dh is None else dh.data_ptr(), 0 if dh is None else _ld(dh),
                                           dx.data_ptr(), max(cols, 1), dw.data_ptr(), _stream(stream))
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_rmsnorm_backward")
    return dx, dw


def _experts(w, name, experts, rows, cols) -> ExpertsStruct:
    import torch
    data, scale = w
    _check(data, name, 3, torch.float8_e4m3fn)
    _check(scale, name + " scales", 3, torch.float32)
    if tuple(data.shape) != (experts, rows, cols):
        raise ValueError(f"{name} must have shape {(experts, rows, cols)}, got {tuple(data.shape)}")
    if tuple(scale.shape) != (experts, -(-rows // 128), -(-cols // 128)):
        raise ValueError(f"{name} scales must have shape {(experts, -(-rows // 128), -(-cols // 128))}, got {tuple(scale.shape)}")
    return ExpertsStruct(data.data_ptr(), data.stride(1), data.stride(0), scale.data_ptr(), max(scale.stride(1), 1), scale.stride(0))


def moe_fp8(x: Fp8Matrix, logits, top_k, gate, up, down, *, renormalize=True, out=None, out_dtype=None, stream=None):
    """A mixture-of-experts layer for a few tokens (sgemm_fp8_moe): for each row t of x the sum over the `top_k` experts with
    the largest logits (ties: lowest index) of their softmax weight times down_e (silu(gate_e x_t) * (up_e x_t)).

    x: E4M3 with groups of (1, 128), at most 64 rows; logits: float32 [tokens, experts]; gate and up: (codes [experts, inner,
    hidden], scales [experts, inner / 128, hidden / 128]) with groups of 128 x 128, down: [experts, hidden, inner].  The
    weights are divided by their sum over the chosen experts with renormalize=True.  Returns bfloat16 unless out_dtype or
    out says otherwise."""
    import torch
    _check(logits, "logits", 2, torch.float32)
    tokens, hidden = x.data.shape
    experts, inner = gate[0].shape[:2]
    if tuple(logits.shape) != (tokens, experts):
        raise ValueError("logits must have one value per token and expert")
    g = _experts(gate, "gate", experts, inner, hidden)
    u = _experts(up, "up", experts, inner, hidden)
    d = _experts(down, "down", experts, hidden, inner)
    y = out if out is not None else _empty((tokens, hidden), out_dtype or torch.bfloat16, x.data, stream)
    if tuple(y.shape) != (tokens, hidden):
        raise ValueError("out has the wrong shape")
    t = _type(_check(y, "out").dtype)
    if out_dtype is not None and y.dtype != out_dtype:
        raise TypeError(f"out is {y.dtype}, not {out_dtype}")
    st = _lib().sgemm_fp8_moe(tokens, hidden, inner, experts, top_k, x._struct, logits.data_ptr(), _ld(logits), 1 if renormalize else 0,
                              g, u, d, y.data_ptr(), _ld(y), t, _stream(stream))
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_moe")
    return y
