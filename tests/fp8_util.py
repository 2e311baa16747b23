"""Helpers of the 8-bit tests: the codes' values and rounding written out in numpy, groups, and
references in 64 bits."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # unit roundoff of float32
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
TINY = np.float32(2.0 ** -126)


def code_values(fmt: str) -> np.ndarray:
    """The value of each of the 256 codes: sign, exponent (4 or 5 bits), fraction (3 or 2 bits)."""
    out = np.empty(256)
    ebits, fbits, bias = (4, 3, 7) if fmt == "e4m3" else (5, 2, 15)
    for c in range(256):
        e, f = (c >> fbits) & ((1 << ebits) - 1), c & ((1 << fbits) - 1)
        v = f * 2.0 ** (1 - bias - fbits) if e == 0 else (1 + f / (1 << fbits)) * 2.0 ** (e - bias)
        if fmt == "e4m3" and (c & 0x7F) == 0x7F:
            v = np.nan
        if fmt == "e5m2" and e == 31:
            v = np.inf if f == 0 else np.nan
        out[c] = -v if c & 0x80 else v
    return out


def round_codes(t: np.ndarray, fmt: str) -> np.ndarray:
    """The value of the code nearest to t (ties to the even code, at most the largest finite one); NaN for non-finite t."""
    vals = code_values(fmt)[:128]
    pos = vals[np.isfinite(vals)]                    # ascending; the index is the code
    a = np.abs(t.astype(np.float64))
    a = np.where(np.isfinite(a), a, 0.0)
    hi = np.clip(np.searchsorted(pos, a), 0, len(pos) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    pick = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    pick = np.where(a >= pos[-1], len(pos) - 1, pick)
    v = np.copysign(pos[pick], t)
    return np.where(np.isfinite(t), v, np.nan)


def groups_of(shape, block):
    return -(-shape[0] // block[0]), -(-shape[1] // block[1])


def spread(scale: np.ndarray, block, shape) -> np.ndarray:
    return np.repeat(np.repeat(scale, block[0], 0)[: shape[0]], block[1], 1)[:, : shape[1]]


def quantize_ref(x: np.ndarray, block, fmt: str):
    """Scales (float32) and code values of float32 x, each operation rounded as the definition says."""
    gr, gc = groups_of(x.shape, block)
    s = np.empty((gr, gc), np.float32)
    for i in range(gr):
        for j in range(gc):
            g = np.abs(x[i * block[0]:(i + 1) * block[0], j * block[1]:(j + 1) * block[1]])
            g = g[np.isfinite(g)]
            amax = np.float32(g.max() if g.size else 0.0)
            s[i, j] = max(np.float32(amax / np.float32(TOP[fmt])), TINY)
    inv = np.float32(1.0) / s
    with np.errstate(all="ignore"):
        t = x.astype(np.float32) * spread(inv, block, x.shape)
    return s, round_codes(np.where(np.isfinite(x), t, np.nan), fmt)


def values(m) -> np.ndarray:
    """Code values of an Fp8Matrix as float64."""
    import torch
    fmt = "e4m3" if m.data.dtype == torch.float8_e4m3fn else "e5m2"
    return code_values(fmt)[m.data.contiguous().view(torch.uint8).cpu().numpy()]


def dequantize(m) -> np.ndarray:
    return values(m) * spread(m.scale.cpu().numpy().astype(np.float64), m.block, tuple(m.shape))


def strided(x, pad, offset=0):
    """A CUDA copy of the 2-D tensor x whose rows lie `pad` elements further apart, `offset` elements past an
    aligned base; the gaps hold NaN."""
    import torch
    rows, cols = x.shape
    buf = torch.full((rows * (cols + pad) + offset,), float("nan"), dtype=x.dtype, device="cuda")
    v = buf[offset:].view(rows, cols + pad)[:, :cols] if rows * (cols + pad) else buf[offset:].view(rows, cols + pad)
    v.copy_(x)
    return v
