"""The 8-bit operators through the bounds-checking build (libsgemm_debug.so): every kernel on small, odd, ragged and
strided operands records no index outside its buffer and gives the normal build's results, bit for bit."""
import ctypes
import itertools

import pytest

import sgemm_row_major_gb300 as sg
from fp8_util import strided
from sgemm_row_major_gb300 import fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbg():
    from sgemm_row_major_gb300 import build
    build.build(debug=True)
    fp8._lib()
    return fp8._declare(sg.load_debug())


@pytest.fixture
def both(dbg, monkeypatch):
    """both(call): the tensors that call() returns are the same from both builds, and the debug build has nothing to report."""
    import torch

    def flat(x):
        if isinstance(x, sg.Fp8Matrix):
            x = (x.data.view(torch.uint8), x.scale)
        return [t for e in x for t in flat(e)] if isinstance(x, tuple) else [] if x is None else [x]

    def run(call, what=None):
        want = flat(call())
        with monkeypatch.context() as m:
            m.setattr(fp8, "_functions", dbg)
            got = flat(call())
        site, off = ctypes.c_uint(0), ctypes.c_longlong(0)
        st = dbg.sgemm_sync_status(None)
        assert dbg.sgemm_bounds_report(ctypes.byref(site), ctypes.byref(off)) == 0
        assert (st, site.value, off.value) == (0, 0, 0), what
        assert len(want) == len(got) and all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
                                             for a, b in zip(want, got)), what
    return run


@pytest.fixture
def force(dbg):
    """force(kernel, tile, split) in both builds, for one test."""
    def set_(variant="AUTO", tile=0, split=0):
        sg.sgemm_fp8_set_override(variant, tile, split)
        assert dbg.sgemm_fp8_set_override({"AUTO": 0, "FP8_PAIR": 32, "FP8_SHORT": 33}[variant], tile, split) == 0
    yield set_
    set_()


def rows(n, cols, dtype, pad, offset, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return strided(torch.randn(n, cols, generator=g, device="cuda").to(getattr(torch, dtype)), pad, offset)


SHAPES = [(1, 1), (3, 7), (130, 129), (200, 328), (5, 1000), (300, 128)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
def test_quantiser(both, dtype, pad, offset):
    for (n, cols), block in itertools.product(SHAPES, fp8.GROUPS):
        x = rows(n, cols, dtype, pad, offset, n + cols)
        both(lambda: sg.quantize_fp8(x, block), (n, cols, block))
    x[0, 0] = float("inf")  # (a tile that is done again)
    both(lambda: sg.quantize_fp8(x))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
def test_norm_and_gradient(both, dtype, pad, offset):
    import torch
    for n, cols in SHAPES + [(400, 520), (3, 8192), (2, 8200), (2, 33000), (700, 4096)]:
        x, r, dy, dh = (rows(n, cols, dtype, pad, offset, s) for s in range(4))
        w = torch.ones(cols, dtype=x.dtype, device="cuda")
        both(lambda: tuple(sg.rmsnorm_fp8(x, w, 1e-6, r, y=True)), (n, cols))
        both(lambda: tuple(sg.rmsnorm_fp8(x, w)), (n, cols))
        out = sg.rmsnorm_fp8(x, w, 1e-6, r)
        both(lambda: sg.rmsnorm_fp8_backward(dy, out.h, w, out.rstd, dh), (n, cols))
        both(lambda: sg.rmsnorm_fp8_backward(dy, x, w, out.rstd), (n, cols))


@pytest.mark.parametrize("kernel,tile,split", [("FP8_PAIR", 64, 0), ("FP8_PAIR", 128, 0), ("FP8_PAIR", 256, 0), ("FP8_SHORT", 16, 1),
                                               ("FP8_SHORT", 32, 2), ("FP8_SHORT", 64, 4), ("FP8_SHORT", 128, 8)])
@pytest.mark.parametrize("ops", ["NN", "NT", "TN", "TT"])
def test_product(both, force, kernel, tile, split, ops):
    import torch
    force(kernel, tile, split)
    for (M, N, K), gb in itertools.product(((1, 1, 1), (5, 300, 77), (300, 7, 260), (530, 280, 1200)), (1, 128)):
        a = rows(*((K, M) if ops[0] == "T" else (M, K)), "float32", 0, 0, 1)
        b = rows(*((K, N) if ops[1] == "N" else (N, K)), "float32", 0, 0, 2)
        a = sg.quantize_fp8(a, (128, 1) if ops[0] == "T" else (1, 128))
        b = sg.quantize_fp8(b, (128, 128) if gb == 128 else (128, 1) if ops[1] == "N" else (1, 128))
        packed = sg.Fp8Matrix(a.data.contiguous(), a.scale, a.block)  # (copied to aligned rows first)
        for dtype, pad, beta in (("float32", 0, 0.0), ("bfloat16", 8, 0.0), ("float32", 4, 1.0), ("bfloat16", 3, 1.0), ("bfloat16", 8, -1.0)):
            c = rows(M, N, dtype, pad, 0, 3)
            d = torch.zeros_like(strided(c, pad))
            both(lambda: sg.matmul_fp8(a if pad else packed, b, c, ops[0], ops[1], 1.5, beta, out=strided(d, pad)), (M, N, K, gb, dtype, pad, beta))
    both(lambda: sg.matmul_fp8(a, b, c, ops[0], ops[1], 0.0, 2.0, out=strided(d, pad)))


@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 16, 16), (1, 64, 8, 512, 256), (7, 16, 3, 400, 336), (17, 40, 6, 656, 64), (64, 128, 8, 256, 128),
                                       (5, 1000, 16, 128, 128), (33, 26, 4, 2048, 1024)])
def test_experts(both, T, E, k, H, I):
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)

    def stack(n, cols):
        codes = torch.randint(0, 256, (E, n, cols + 16), generator=g, device="cuda", dtype=torch.uint8)[..., :cols] & 0xB7
        scale = torch.rand(E, -(-n // 128), -(-cols // 128) + 1, generator=g, device="cuda")[..., :-1] * 0.1
        wide = torch.zeros(E, n, cols + 16, dtype=torch.uint8, device="cuda")[..., :cols]
        wide.copy_(codes)
        return wide.view(torch.float8_e4m3fn), scale
    x = sg.quantize_fp8(rows(T, H, "bfloat16", 0, 0, 1))
    logits = rows(T, E, "float32", 3, 0, 2)
    gate, up, down = stack(I, H), stack(I, H), stack(H, I)
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.zeros(T, H, dtype=dtype, device="cuda")
        both(lambda: sg.moe_fp8(x, logits, k, gate, up, down, out=strided(y, 3)))
