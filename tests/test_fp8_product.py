"""The block-scaled 8-bit product (sgemm_fp8) against the formula in 64 bits.

Bound per element: (K + 2) u (|alpha| sum|a b| + |beta c|) with u = 2^-24, and half a unit in the last
place of D's type.  Codes that are small whole numbers with power-of-two scales give the exact result."""
import numpy as np
import pytest

import sgemm_row_major_gb300 as sg
from fp8_util import U, code_values, dequantize, groups_of, spread

FAKE = 1 << 20
OPS = ["NN", "NT", "TN", "TT"]
KERNELS = ["FP8_PAIR", "FP8_SHORT"]


@pytest.fixture
def force():
    """force(kernel, tile, split) for one test."""
    yield sg.sgemm_fp8_set_override
    sg.sgemm_fp8_set_override("AUTO")


def matrix(rows, cols, block, fmt, seed, pad=0, offset=0, exact=False):
    """An Fp8Matrix of random codes and scales; the bytes between its rows are NaN codes."""
    import torch
    rng = np.random.default_rng(seed)
    vals = code_values(fmt)
    if exact:
        usable = np.flatnonzero(np.isin(vals, [-3.0, -2.0, -1.0, 0.0, 1.0, 2.0]))
        scale = np.exp2(rng.integers(-2, 3, groups_of((rows, cols), block)))
    else:  # normal values up to a few units
        usable = np.flatnonzero((np.abs(vals) <= 8) & (np.abs(vals) >= 2.0 ** -6))
        scale = rng.uniform(0.25, 2.0, groups_of((rows, cols), block))
    ld = cols + pad
    buf = np.full(rows * ld + offset, 0x7F, np.uint8)
    codes = rng.choice(usable, (rows, cols)).astype(np.uint8)
    buf[offset:].reshape(rows, ld)[:, :cols] = codes
    t = torch.from_numpy(buf).cuda()[offset:].view(rows, ld)[:, :cols]
    return sg.Fp8Matrix(t.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2),
                        torch.from_numpy(scale.astype(np.float32)).cuda(), block)


def operands(ops, M, N, K, ga, gb, fa, fb, seed, pad=(0, 0), offset=0, exact=False):
    """A and B with groups of 128 along k: ga / gb tell the group's extent along the other dimension."""
    ta, tb = ops[0] == "T", ops[1] == "T"
    block = lambda along_rows, g: (128, g) if along_rows else (g, 128)  # noqa: E731
    a = matrix(*((K, M) if ta else (M, K)), block(ta, ga), fa, seed, pad[0], offset, exact)
    b = matrix(*((N, K) if tb else (K, N)), block(not tb, gb), fb, seed + 1, pad[1], offset, exact)
    return a, b


def reference(ops, a, b, alpha=1.0, beta=0.0, c=None):
    A, B = dequantize(a), dequantize(b)
    A, B = (A.T if ops[0] == "T" else A), (B.T if ops[1] == "T" else B)
    ref, mag = alpha * (A @ B), abs(alpha) * (np.abs(A) @ np.abs(B))
    if c is not None and beta != 0:
        ref, mag = ref + beta * c, mag + np.abs(beta * c)
    return ref, mag, A.shape[1]


def check(got, ref, mag, K, bf16=False, what=""):
    import torch
    g = got.double().cpu().numpy()
    tol = (K + 2) * U * mag + (2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) if bf16 else 0.0)
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4])
    assert sg.sgemm_sync_status(torch.cuda.current_stream()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("ops", OPS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (16, 128, 128), (5, 7, 3), (300, 520, 1000), (129, 1000, 77), (513, 80, 640)])
def test_exact_on_whole_numbers(force, kernel, ops, M, N, K):
    """Every partial sum is a small multiple of a power of two: equal bit for bit, every layout and kernel."""
    force(kernel)
    for ga, gb in ((1, 128), (1, 1), (128, 128), (128, 1)):
        a, b = operands(ops, M, N, K, ga, gb, "e4m3", "e5m2", M + N + K, exact=True)
        ref, _, _ = reference(ops, a, b)
        got = sg.matmul_fp8(a, b, transA=ops[0], transB=ops[1]).cpu().numpy()
        assert np.array_equal(got, ref), (ga, gb, np.argwhere(got != ref)[:4], got[got != ref][:4], ref[got != ref][:4])


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("ops", OPS)
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_formats(force, kernel, ops, fa, fb):
    force(kernel)
    for ga, gb in ((1, 128), (1, 1)):
        a, b = operands(ops, 200, 328, 900, ga, gb, fa, fb, 5)
        ref, mag, K = reference(ops, a, b, 1.5)
        check(sg.matmul_fp8(a, b, transA=ops[0], transB=ops[1], alpha=1.5), ref, mag, K)


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [64, 128, 256])
def test_pair_tiles(force, tile):
    """Every tile width, with column blocks that begin inside a tile, B in both orders and with both groupings."""
    force("FP8_PAIR", tile)
    for ops, gb in (("NT", 128), ("NN", 128), ("TN", 1), ("NT", 1)):
        a, b = operands(ops, 530, 1100, 700, 1, gb, "e4m3", "e4m3", tile)
        ref, mag, K = reference(ops, a, b)
        check(sg.matmul_fp8(a, b, transA=ops[0], transB=ops[1]), ref, mag, K, what=(ops, gb))


@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("tile", [64, 128, 256])
@pytest.mark.parametrize("K", [128, 400])
def test_many_short_tiles_per_cluster(force, tile, bf16, K):
    """Tiles that follow one another faster than the last ones are written."""
    import torch
    force("FP8_PAIR", tile)
    M, N = 20000, 512
    a, b = operands("NT", M, N, K, 1, 128, "e4m3", "e4m3", 17)
    A = a.data.double() * a.scale.double().repeat_interleave(128, 1)[:, :K]
    B = b.data.double() * b.scale.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    ref, mag = A @ B.T, A.abs() @ B.abs().T
    for _ in range(3):
        got = sg.matmul_fp8(a, b, transB="T", out_dtype=torch.bfloat16 if bf16 else torch.float32)
        bad = (got.double() - ref).abs() > (K + 2) * U * mag + (2.0 ** -8 * ref.abs() if bf16 else 0.0)
        assert not bool(bad.any()), bad.nonzero()[:4]


@pytest.mark.gpu
@pytest.mark.parametrize("split", [1, 2, 4, 8])
@pytest.mark.parametrize("M,N,K", [(1, 300, 128), (3, 4096, 1536), (40, 500, 1000), (128, 257, 2048), (700, 33, 900), (260, 130, 520)])
def test_short_splits(force, split, M, N, K):
    """K shared by clusters, some CTAs without any groups; both orientations; more than one tile of the short side."""
    force("FP8_SHORT", 0, split)
    for ops, gb in (("NT", 128), ("NN", 128), ("TN", 1)):
        a, b = operands(ops, M, N, K, 1, gb, "e4m3", "e4m3", split)
        ref, mag, _ = reference(ops, a, b)
        got = sg.matmul_fp8(a, b, transA=ops[0], transB=ops[1])
        check(got, ref, mag, K, what=(ops, gb))
        assert bool((sg.matmul_fp8(a, b, transA=ops[0], transB=ops[1]) == got).all())


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [16, 32, 64, 128])
def test_short_tiles(force, tile):
    force("FP8_SHORT", tile, 2)
    for ops in OPS:
        a, b = operands(ops, 150, 1000, 600, 1, 128, "e4m3", "e5m2", tile)
        ref, mag, K = reference(ops, a, b)
        check(sg.matmul_fp8(a, b, transA=ops[0], transB=ops[1]), ref, mag, K, what=ops)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("ldc_pad", [0, 8, 3])
def test_alpha_beta_types_and_strides(force, kernel, bf16, ldc_pad):
    """C in place and D elsewhere, padded rows (vectors or single elements), the padding untouched."""
    import torch
    force(kernel)
    M, N, K = 270, 200, 333
    t = torch.bfloat16 if bf16 else torch.float32
    a, b = operands("NT", M, N, K, 1, 128, "e4m3", "e4m3", 21)
    base = torch.randn(M, N + ldc_pad, generator=torch.Generator().manual_seed(1)).to(t).cuda()
    c = base.clone()[:, :N]
    ref, mag, _ = reference("NT", a, b, -0.75, 2.0, c.double().cpu().numpy())
    d = torch.full((M, N + ldc_pad + 1), 7.0, dtype=t, device="cuda")
    got = sg.matmul_fp8(a, b, c, "N", "T", -0.75, 2.0, out=d[:, :N])
    check(got, ref, mag, K, bf16)
    assert bool((d[:, N:] == 7.0).all()) and torch.equal(c, base[:, :N])
    whole = base.clone()
    check(sg.matmul_fp8(a, b, whole[:, :N], "N", "T", -0.75, 2.0), ref, mag, K, bf16)
    assert torch.equal(whole[:, N:], base[:, N:])


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,tile", [("FP8_PAIR", 64), ("FP8_PAIR", 128), ("FP8_PAIR", 256), ("FP8_SHORT", 0)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("gb", [1, 128])
def test_nothing_is_written_beside_d(force, kernel, tile, bf16, gb):
    """D as columns of a wider matrix whose rows are aligned, at every width modulo 16 bytes: its neighbours on both sides,
    and what lies behind the last row, keep their values."""
    import torch
    force(kernel, tile)
    t = torch.bfloat16 if bf16 else torch.float32
    for M, N in [(150, n) for n in (1, 2, 3, 5, 6, 7, 31, 33, 100, 129, 255, 257, 300, 514, 515, 516, 517, 518, 519)] + [(1, 130), (700, 61)]:
        K = 160
        a, b = operands("NT", M, N, K, 1, gb, "e4m3", "e4m3", N)
        ref, mag, _ = reference("NT", a, b)
        ld = -(-N // 8) * 8 + 16
        big = torch.full((M + 1, ld), 7.0, dtype=t, device="cuda")
        d = big[:M, 8:8 + N]
        for beta in (0.0, 1.0):
            big[:M, 8:8 + N] = 3.0
            c = d if beta else None
            got = sg.matmul_fp8(a, b, c, "N", "T", 1.0, beta, out=d)
            check(got, ref + 3.0 * beta, mag + 3.0 * beta, K, bf16, what=(M, N, beta))
            assert bool((big[:M, :8] == 7.0).all()) and bool((big[:M, 8 + N:] == 7.0).all()) and bool((big[M] == 7.0).all()), (M, N, beta)


@pytest.mark.gpu
@pytest.mark.parametrize("ops", OPS)
@pytest.mark.parametrize("pad,offset", [((16, 32), 0), ((0, 0), 0), ((3, 5), 0), ((16, 16), 1)])
def test_alignment(ops, pad, offset):
    """Codes with any row stride and base: those TMA cannot read are copied to aligned rows first."""
    for M, N, K in ((300, 333, 501), (9, 400, 501)):
        a, b = operands(ops, M, N, K, 1, 128, "e4m3", "e4m3", 31, pad, offset)
        ref, mag, _ = reference(ops, a, b)
        check(sg.matmul_fp8(a, b, transA=ops[0], transB=ops[1]), ref, mag, K)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
def test_special_values(force, kernel):
    """A NaN code, an infinity, a NaN or infinite scale reach the elements whose sums they enter, and no others."""
    import torch
    force(kernel)
    a, b = operands("NT", 160, 200, 300, 1, 128, "e5m2", "e4m3", 41)
    codes = a.data.view(torch.uint8)
    codes[3, 7] = 0x7F        # NaN
    codes[5, 290] = 0x7C      # +Inf
    codes[6, 10], codes[6, 11] = 0x7C, 0xFC
    b.data.view(torch.uint8)[:, 10:12] = 0x38  # 1.0 against the infinities of row 6
    a.scale[8, 1] = float("nan")
    with np.errstate(all="ignore"):
        ref, mag, K = reference("NT", a, b)
    a.scale[9, 2] = float("inf")  # times the group's inner sum: an infinity of either sign
    g = sg.matmul_fp8(a, b, transB="T").cpu().numpy()
    assert np.isinf(g[9]).all()
    g[9] = ref[9]
    assert np.array_equal(np.isnan(g), np.isnan(ref)) and np.array_equal(np.isinf(g), np.isinf(ref))
    assert np.array_equal(np.sign(g[np.isinf(g)]), np.sign(ref[np.isinf(ref)]))
    fine = np.isfinite(ref)
    assert np.all(np.abs(g[fine] - ref[fine]) <= (K + 2) * U * mag[fine])
    assert np.isnan(g[[3, 6, 8]]).all() and fine[[0, 4, 7, 10]].all()


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("fb", ["e4m3", "e5m2"])
def test_whole_range_of_codes(force, kernel, fa, fb):
    """Codes of every finite value, and sums in which the product of the largest code with the smallest subnormal one leads.
    A product of codes m 2^e is aligned by e, and a subnormal code's e is the smallest normal one's, so the bound counts such
    a code as the smallest normal one (the sums of magnitudes alone were exceeded by a third)."""
    import torch
    force(kernel)
    least, rng = {"e4m3": 2.0 ** -6, "e5m2": 2.0 ** -14}, np.random.default_rng(101)
    for K, lead, positive in [(K, lead, positive) for K in (2, 3, 4, 8, 16, 40, 128, 300) for lead in (0, 1, 2) for positive in (False, True)]:
        codes = []
        for i, fmt in enumerate((fa, fb)):
            v = code_values(fmt)
            usable = np.flatnonzero(np.isfinite(v) & ((np.abs(v) < 2.0 ** -3) if lead else True) & (np.signbit(v) <= (not positive)))
            c = rng.choice(usable, (150, K)).astype(np.uint8)
            if lead:
                c[:, 0] = np.nanargmax(np.where(np.isfinite(v), v, np.nan)) if lead == i + 1 else 1  # the largest one, 1: the smallest
            codes.append(c)
        ms, vs, ws = [], [], []
        for c, fmt in zip(codes, (fa, fb)):
            buf = torch.from_numpy(np.pad(c, ((0, 0), (0, -K % 16)))).cuda()[:, :K]
            ms.append(sg.Fp8Matrix(buf.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2), torch.ones(150, -(-K // 128), device="cuda")))
            vs.append(code_values(fmt)[c])
            ws.append(np.where(vs[-1] == 0, 0.0, np.maximum(np.abs(vs[-1]), least[fmt])))
        check(sg.matmul_fp8(*ms, transB="T"), vs[0] @ vs[1].T, ws[0] @ ws[1].T, K, what=(K, lead, positive))


@pytest.mark.gpu
def test_wide_range_of_scales():
    """Scales from the smallest to large ones: products of two scales that FP32 holds."""
    import torch
    a, b = operands("NT", 130, 140, 512, 1, 128, "e4m3", "e4m3", 51)
    a.scale[:, 0], a.scale[:, 1] = 2.0 ** -126, 2.0 ** 60
    b.scale[:, 1] = 2.0 ** -60
    b.scale[:, 0] = 2.0 ** 100
    ref, mag, K = reference("NT", a, b)
    check(sg.matmul_fp8(a, b, transB="T"), ref, mag, K)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,tile", [("FP8_PAIR", 64), ("FP8_PAIR", 256), ("FP8_SHORT", 16), ("FP8_SHORT", 64), ("FP8_SHORT", 128)])
@pytest.mark.parametrize("ops,ga,gb", [("NT", 1, 128), ("TN", 1, 1), ("NN", 128, 128), ("TT", 128, 1)])
@pytest.mark.parametrize("swap", [False, True])
def test_each_scale_may_be_extreme(force, kernel, tile, ops, ga, gb, swap):
    """Scales from 2^-126 to 2^120 on either side whose products are ordinary.  A group's sum times one of them alone would
    be beyond FP32 (codes up to 448), or lose its bits (three products of codes of at most 7 2^-9)."""
    import torch
    force(kernel, tile)
    for M, N, K in ((130, 140, 200), (140, 130, 200), (130, 140, 3), (140, 130, 3)):  # either side along the tensor core's rows
        a, b = operands(ops, M, N, K, ga, gb, "e4m3", "e4m3", 91)
        for m, down in ((a, ops[0] == "T"), (b, ops[1] == "N")):  # k along dimension 0 where `down`
            codes, scale = m.data.view(torch.uint8), m.scale if down else m.scale.T
            if K == 3:
                codes.bitwise_and_(0x87)
            else:
                codes.bitwise_or_(0x70)
                codes[(codes & 0x7F) == 0x7F] = 0x7E
            low = (m is a) != swap
            scale[0].mul_(2.0 ** -125 if low else 2.0 ** 119)
            scale[1:].mul_(2.0 ** 119 if low else 2.0 ** -125)
        ref, mag, _ = reference(ops, a, b)
        check(sg.matmul_fp8(a, b, transA=ops[0], transB=ops[1]), ref, mag, K, what=(M, N, K))


@pytest.mark.gpu
def test_nothing_is_read_that_need_not_be():
    import torch
    a, b = operands("NT", 20, 30, 128, 1, 128, "e4m3", "e4m3", 61)
    c = torch.full((20, 30), float("nan"), device="cuda")
    assert bool(torch.isfinite(sg.matmul_fp8(a, b, c, "N", "T", 1.0, 0.0)).all())
    a.data.view(torch.uint8).fill_(0x7F)
    c.fill_(3.0)
    assert bool((sg.matmul_fp8(a, b, c, "N", "T", 0.0, 0.5) == 1.5).all())
    e = sg.Fp8Matrix(a.data[:, :0], a.scale[:, :0])
    f = sg.Fp8Matrix(b.data[:, :0], b.scale[:1, :0], (128, 128))
    assert bool((sg.matmul_fp8(e, f, c, "N", "T", 1.0, 2.0) == 3.0).all())
    assert sg.matmul_fp8(sg.Fp8Matrix(a.data[:0], a.scale[:0]), b, transB="T").shape == (0, 30)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Codes and results more than 2^31 elements from their base."""
    import torch
    M, N, K, ld = 60000, 16, 200, 40000
    torch.cuda.empty_cache()
    codes = torch.zeros(M * ld, dtype=torch.uint8, device="cuda").view(M, ld)[:, :K]
    src, b = operands("NT", M, N, K, 1, 128, "e4m3", "e4m3", 71)
    codes.copy_(src.data.view(torch.uint8))
    a = sg.Fp8Matrix(codes.view(torch.float8_e4m3fn), src.scale)
    want = sg.matmul_fp8(src, b, transB="T", out_dtype=torch.bfloat16)
    d = torch.zeros(M * ld, dtype=torch.bfloat16, device="cuda").view(M, ld)[:, :N]
    for kernel in KERNELS:
        sg.sgemm_fp8_set_override(kernel)
        try:
            d.zero_()
            sg.matmul_fp8(a, b, transB="T", out=d)
        finally:
            sg.sgemm_fp8_set_override("AUTO")
        diff = (d.float() - want.float()).abs()
        assert bool((diff <= 2.0 ** -7 * want.float().abs() + 1e-4).all())
    ref, mag, _ = reference("NT", src, b)
    check(want, ref, mag, K, True)


@pytest.mark.gpu
def test_training_step_of_a_layer():
    """Forward, input gradient and weight gradient of one layer from one quantised weight matrix: the three
    layouts read the same codes."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    T, I, O = 300, 400, 272
    x, w, dy = (torch.randn(r, c, generator=g, device="cuda") for r, c in ((T, I), (O, I), (T, O)))
    qx, qw = sg.quantize_fp8(x), sg.quantize_fp8(w, (128, 128))
    qdy = sg.quantize_fp8(dy, format="e5m2")
    ref, mag, K = reference("NT", qx, qw)
    check(sg.matmul_fp8(qx, qw, transB="T"), ref, mag, K)
    ref, mag, K = reference("NN", qdy, qw)
    check(sg.matmul_fp8(qdy, qw), ref, mag, K)
    cdy, cx = sg.quantize_fp8(dy, (128, 1), "e5m2"), sg.quantize_fp8(x, (128, 1))
    dw = torch.randn(O, I, generator=g, device="cuda")
    ref, mag, K = reference("TN", cdy, cx, 1.0, 1.0, dw.double().cpu().numpy())
    check(sg.matmul_fp8(cdy, cx, dw, "T", "N", 1.0, 1.0), ref, mag, K)


@pytest.mark.gpu
def test_graph_and_streams():
    import torch
    for M in (3, 300):
        a, b = operands("NT", M, 500, 700, 1, 128, "e4m3", "e4m3", 81, pad=(3, 16))  # A goes through the workspace
        want = sg.matmul_fp8(a, b, transB="T")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = sg.matmul_fp8(a, b, transB="T", stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = sg.matmul_fp8(a, b, transB="T")
        a.scale.mul_(2.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, 2 * want)


# ------------------------------------------------------------------ host logic

def struct(rows, cols, block=(1, 128), fmt=0, data=FAKE, scale=FAKE, ld=None, lds=None):
    from sgemm_row_major_gb300.fp8 import MatrixStruct
    gc = -(-cols // block[1])
    return MatrixStruct(data, max(cols, 1) if ld is None else ld, scale, max(gc, 1) if lds is None else lds, fmt, *block)


def plan(ops, M, N, K, a=None, b=None, sm=152, **kw):
    ta, tb = ops[0] == "T", ops[1] == "T"
    a = a or struct(*((K, M) if ta else (M, K)), (128, 1) if ta else (1, 128))
    b = b or struct(*((N, K) if tb else (K, N)), (128, 128))
    args = dict(alpha=1.0, beta=0.0, C=None, ldc=1, D=FAKE, ldd=N, type=0)
    args.update(kw)
    return sg.sgemm_fp8_plan(ops[0], ops[1], M, N, K, args["alpha"], a, b, args["beta"], args["C"], args["ldc"], args["D"],
                             args["ldd"], args["type"], sm)


def test_planner():
    p = plan("NT", 1, 4096, 4096)
    assert p["variant_name"] == "FP8_SHORT" and p["tile_n"] == 16 and p["split_k"] in (2, 4, 8)
    assert p["grid_x"] == 32 * p["split_k"] and p["workspace_bytes"] == 0
    p = plan("NT", 8192, 8192, 8192)
    assert p["variant_name"] == "FP8_PAIR" and p["tile_m"] == 256 and p["tile_n"] % 32 == 0 and p["grid_x"] <= 152
    assert plan("NT", 4, 300, 100)["workspace_bytes"] == 512 + 33792  # both copied to rows of 112 bytes, in pieces of 256
    assert plan("NT", 0, 8, 8)["variant_name"] == "NONE" and plan("NT", 8, 8, 0)["variant_name"] == "SCALE"
    assert plan("NT", 8, 8, 8, alpha=0.0)["variant_name"] == "SCALE"


def test_one_stored_row_is_read_in_place():
    """A single aligned row needs no copy whatever its length and stride: the operand of a decoding step."""
    w = struct(4096, 4095, (128, 128), ld=4096)
    for ld in (4095, 4096, 4111):
        p = plan("NT", 1, 4096, 4095, a=struct(1, 4095, ld=ld), b=w)
        assert p["workspace_bytes"] == 0 and p["kernel_launches"] == 1, ld
    assert plan("TN", 301, 40, 1, a=struct(1, 301, (128, 1)), b=struct(1, 40, (128, 128), ld=41))["workspace_bytes"] == 0
    assert plan("NT", 1, 4096, 4095, a=struct(1, 4095, data=FAKE + 1), b=w)["workspace_bytes"] == 4096
    assert plan("NT", 2, 4096, 4095, a=struct(2, 4095), b=w)["workspace_bytes"] == 2 * 4096


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
def test_one_stored_row_of_any_length(force, kernel):
    """Rows of odd lengths, read in place; what lies behind them is NaN."""
    force(kernel)
    for ops, M, N, K, pad in (("NT", 1, 300, 501, (11, 11)), ("NN", 1, 304, 127, (3, 0)), ("TN", 301, 40, 1, (5, 9)), ("TT", 33, 1, 1, (2, 7))):
        a, b = operands(ops, M, N, K, 1, 128, "e4m3", "e4m3", 33, pad)
        ref, mag, _ = reference(ops, a, b)
        check(sg.matmul_fp8(a, b, transA=ops[0], transB=ops[1]), ref, mag, K, what=(ops, K))


def test_refusals():
    def refused(code, *a, **kw):
        with pytest.raises(sg.SgemmError) as e:
            plan(*a, **kw)
        assert e.value.status == code
    refused(-1, "XT", 8, 8, 128, a=struct(8, 128), b=struct(8, 128))
    refused(-2, "NX", 8, 8, 128, a=struct(8, 128), b=struct(8, 128))
    refused(-3, "NT", -1, 8, 128, a=struct(8, 128), b=struct(8, 128))
    refused(-4, "NT", 8, -1, 128, a=struct(8, 128), b=struct(8, 128))
    refused(-5, "NT", 8, 8, -1, a=struct(8, 128), b=struct(8, 128))
    for bad in (struct(8, 200, fmt=2), struct(8, 200, (128, 1)), struct(8, 200, (1, 1)), struct(8, 200, data=None), struct(8, 200, scale=None),
                struct(8, 200, scale=FAKE + 2), struct(8, 200, ld=199), struct(8, 200, lds=1), struct(8, 200, (64, 128))):
        refused(-7, "NT", 8, 8, 200, a=bad)
        refused(-8, "NT", 8, 8, 200, b=bad)
    refused(-7, "TT", 8, 8, 200, a=struct(200, 8, (1, 128)))  # k runs down the stored columns: groups must too
    refused(-10, "NT", 8, 8, 128, beta=1.0, ldc=8)
    refused(-11, "NT", 8, 8, 128, beta=1.0, C=FAKE, ldc=7)
    refused(-12, "NT", 8, 8, 128, D=None)
    refused(-12, "NT", 8, 8, 128, D=FAKE + 2)
    refused(-13, "NT", 8, 8, 128, ldd=7)
    refused(-13, "NT", 8, 8, 128, beta=1.0, C=FAKE, ldc=9, ldd=8)  # C in place has one stride
    refused(-14, "NT", 8, 8, 128, type=2)
    refused(4, "NT", 1 << 31, 8, 128)
    for bad in (("FP8_PAIR", 16, 0), ("FP8_PAIR", 96, 0), ("FP8_PAIR", 288, 0), ("FP8_SHORT", 144, 0), ("FP8_SHORT", 48, 0), ("AUTO", 32, 0)):
        with pytest.raises(sg.SgemmError):
            sg.sgemm_fp8_set_override(*bad)
    for bad in (("FP8_PAIR", 0, 2), ("FP8_SHORT", 0, 3)):
        with pytest.raises(sg.SgemmError):
            sg.sgemm_fp8_set_override(*bad)


def test_matrix_refusals():
    import torch
    with pytest.raises(TypeError):
        sg.Fp8Matrix(torch.zeros(4, 4), torch.zeros(4, 1))
    with pytest.raises(TypeError):
        sg.Fp8Matrix(torch.zeros(4, 4, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(4, 1))  # not on the GPU
