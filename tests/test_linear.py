"""Layers and gated blocks on BF16 matrices against their formulas in 64 bits (tolerances: linear_util.py), on every kernel."""
import pytest

import sgemm_row_major_gb300 as sg
from fp8_util import strided
from linear_util import ACTS, check_all, check_kept, close, gated_grad_ref, gated_ref, linear_grad_ref, linear_ref, rounded, values

pytestmark = pytest.mark.gpu

KERNELS = [("AUTO", 0, 0), ("LINEAR_SHORT", 16, 1), ("LINEAR_SHORT", 32, 2), ("LINEAR_SHORT", 64, 4), ("LINEAR_SHORT", 128, 8), ("LINEAR_SHORT", 16, 8),
           ("LINEAR_PAIR", 64, 0), ("LINEAR_PAIR", 128, 0), ("LINEAR_PAIR", 256, 0), ("LINEAR_PAIR", 64, 2), ("LINEAR_PAIR", 128, 5),
           ("LINEAR_PAIR", 256, 32)]
# tokens, inputs, outputs: ones, below and beyond a tile, a fold of 512 and more, odd everything
SHAPES = [(1, 1, 1), (1, 64, 128), (3, 7, 5), (17, 129, 33), (64, 512, 256), (130, 520, 264), (257, 1100, 129), (300, 1304, 713)]


@pytest.fixture
def force():
    yield sg.sgemm_linear_set_override
    sg.sgemm_linear_set_override()


def rand(seed, *shape, std=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()


def done():
    assert sg.sgemm_sync_status() == 0


def options(i):
    """Bias, activation, residual, what is kept and the output's type of case i: every pair of neighbours in turn."""
    import torch
    return i % 2 == 0, ACTS[i % 5], i % 3 != 1, (None, "bf16", "fp8")[i % 3], (torch.bfloat16, torch.float32)[i // 2 % 2]


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: f"{k[0]}{k[1]}_{k[2]}")
def test_linear(force, kernel):
    force(*kernel)
    for i, (T, I, O) in enumerate(SHAPES * 2):
        bias, activation, residual, save, dtype = options(i + KERNELS.index(kernel))
        x, w = rand(i, T, I), rand(i + 1, O, I, std=I ** -0.5)
        b, r = rand(i + 2, 1, O)[0] if bias else None, rand(i + 3, T, O) if residual else None
        got = sg.linear_bf16(x, w, b, activation, r, save=save, out_dtype=dtype)
        ref = linear_ref(x, w, b, activation, r)
        check_all(got, ref, ["y"])
        if save:
            check_kept(got.pre, *ref["pre"], what=f"{T}x{I}x{O} {activation}")
        else:
            assert got.pre is None
    done()


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: f"{k[0]}{k[1]}_{k[2]}")
def test_gated(force, kernel):
    force(*kernel)
    for i, (T, I, O) in enumerate(SHAPES * 2):
        _, _, _, save, _ = options(i + KERNELS.index(kernel))
        activation = ACTS[(i + KERNELS.index(kernel)) % 5]
        x, g, u = rand(i, T, I), rand(i + 1, O, I, std=I ** -0.5), rand(i + 2, O, I, std=I ** -0.5)
        got = sg.gated_bf16(x, g, u, activation, save=save)
        ref = gated_ref(x, g, u, activation)
        check_all(got, ref, ["h"])
        if save:
            for name in ("gate", "up"):
                check_kept(getattr(got, name), *ref[name], what=f"{T}x{I}x{O} {name}")
    done()


def kept_of(v, how):
    return v if how == "bf16" else sg.quantize_fp8(v)


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: f"{k[0]}{k[1]}_{k[2]}")
def test_linear_gradients(force, kernel):
    import torch
    force(*kernel)
    for i, (T, I, O) in enumerate(SHAPES * 2):
        j = i + KERNELS.index(kernel)
        activation, how, x8 = ACTS[j % 5], ("bf16", "fp8")[j // 2 % 2], j % 4 == 3
        dy, x, w = rand(i, T, O, std=0.1), rand(i + 1, T, I), rand(i + 2, O, I, std=O ** -0.5)
        x = sg.quantize_fp8(x) if x8 else x
        pre = kept_of(rand(i + 3, T, O), how) if activation else None
        got = sg.linear_bf16_backward(dy, x, w, pre, activation, dbias=True, dweight_dtype=(torch.bfloat16, torch.float32)[j % 2])
        check_all(got, linear_grad_ref(dy, x, w, pre, activation))
    done()


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: f"{k[0]}{k[1]}_{k[2]}")
def test_gated_gradients(force, kernel):
    import torch
    force(*kernel)
    for i, (T, I, O) in enumerate(SHAPES * 2):
        j = i + KERNELS.index(kernel)
        activation, how, x8 = ACTS[j % 5], ("bf16", "fp8")[j // 2 % 2], j % 4 == 3
        dh, x = rand(i, T, O, std=0.1), rand(i + 1, T, I)
        gate, up = rand(i + 2, O, I, std=O ** -0.5), rand(i + 3, O, I, std=O ** -0.5)
        x = sg.quantize_fp8(x) if x8 else x
        a, b = kept_of(rand(i + 4, T, O), how), kept_of(rand(i + 5, T, O), how)
        got = sg.gated_bf16_backward(dh, x, gate, up, a, b, activation, h=True, dweight_dtype=(torch.bfloat16, torch.float32)[j % 2])
        check_all(got, gated_grad_ref(dh, x, gate, up, a, b, activation))
    done()


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 0), (5, 1), (16, 3)])
@pytest.mark.parametrize("T,I,O", [(1, 77, 130), (5, 256, 96), (70, 333, 300), (530, 200, 257)])
def test_any_rows(T, I, O, pad, offset):
    """Rows of any stride and alignment with NaN between them give what packed copies give, bit for bit, and nothing is
    written between the rows of an output."""
    import torch
    x, w, u, b, r = rand(1, T, I), rand(2, O, I), rand(3, O, I), rand(4, 1, O)[0], rand(5, T, O)
    wide = [strided(v, pad, offset) for v in (x, w, u, r)]
    sx, sw, su, sr = wide
    sb = strided(b[None], 0, offset)[0]
    for dtype in (torch.bfloat16, torch.float32):
        want = sg.linear_bf16(x, w, b, "gelu", r, save="bf16", out_dtype=dtype)
        out = strided(torch.zeros(T, O, dtype=dtype, device="cuda"), pad, offset)
        got = sg.linear_bf16(sx, sw, sb, "gelu", sr, save="bf16", out=out)
        assert got.y is out and torch.equal(got.y, want.y) and torch.equal(got.pre, want.pre)
        whole = out.as_strided((T * (O + pad),), (1,))
        assert int(whole.isnan().sum()) == T * pad
    want = sg.gated_bf16(x, w, u, save="fp8")
    out = strided(torch.zeros(T, O, dtype=torch.bfloat16, device="cuda"), pad, offset)
    got = sg.gated_bf16(sx, sw, su, save="fp8", out=out)
    assert torch.equal(got.h, want.h) and int(out.as_strided((T * (O + pad),), (1,)).isnan().sum()) == T * pad
    for k in ("gate", "up"):
        p, q = getattr(got, k), getattr(want, k)
        assert torch.equal(p.scale, q.scale) and torch.equal(p.data.view(torch.uint8), q.data.view(torch.uint8))
    dy, a = rand(6, T, O), rand(7, T, O)
    sdy, sa = strided(dy, pad, offset), strided(a, pad, offset)
    for activation in (None, "silu"):
        want, got = sg.linear_bf16_backward(dy, x, w, a, activation, dbias=True), sg.linear_bf16_backward(sdy, sx, sw, sa, activation, dbias=True)
        assert all(torch.equal(p, q) for p, q in zip(want, got))
    want, got = sg.gated_bf16_backward(dy, x, w, u, a, r, h=True), sg.gated_bf16_backward(sdy, sx, sw, su, sa, sr, h=True)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    # codes of rows that lie anywhere
    qa, qr, qx = (sg.quantize_fp8(v) for v in (a, r, x))
    move = lambda m: sg.Fp8Matrix(strided_codes(m.data, pad, offset), strided(m.scale, pad, 0))  # noqa: E731
    want = sg.gated_bf16_backward(dy, qx, w, u, qa, qr, h=True)
    got = sg.gated_bf16_backward(dy, move(qx), w, u, move(qa), move(qr), h=True)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    done()


def strided_codes(codes, pad, offset):
    import torch
    rows, cols = codes.shape
    buf = torch.full((rows * (cols + pad) + offset,), 0x7F, dtype=torch.uint8, device="cuda")
    v = buf[offset:].view(rows, cols + pad)[:, :cols]
    v.copy_(codes.view(torch.uint8))
    return v.view(torch.float8_e4m3fn)


@pytest.mark.parametrize("kernel", [("LINEAR_SHORT", 16, 2), ("LINEAR_PAIR", 128, 0), ("LINEAR_PAIR", 256, 0)], ids=str)
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_residual_in_place(force, kernel, pad):
    import torch
    force(*kernel)
    T, I, O = 300, 700, 520
    x, w, r = rand(1, T, I), rand(2, O, I), rand(3, T, O)
    want = sg.linear_bf16(x, w, None, "silu", r).y
    stream = strided(r, pad)
    got = sg.linear_bf16(x, w, None, "silu", stream, out=stream).y
    assert got is stream and torch.equal(got, want)
    done()


def test_shared_k_as_chosen():
    """Long K and few tiles, where the planner shares K: residuals in place and kept values with rows at any alignment, products
    with and without shares in one launch, and two captured calls whose workspaces are in use at the same time."""
    import torch
    T, I, O = 4, 15527, 108
    assert sg.sgemm_linear_plan(T, O, I)["kernel_launches"] == 2 and sg.sgemm_linear_plan(1024, 1024, 16384)["split_k"] > 1
    x, w, b, r = rand(1, T, I), rand(2, O, I, std=I ** -0.5), rand(3, 1, O)[0], rand(4, T, O)
    ref = linear_ref(x, w, b, "gelu", r)
    want = sg.linear_bf16(x, w, b, "gelu", r, save="bf16")
    check_all(want, ref, ["y"])
    check_kept(want.pre, *ref["pre"])
    for pad, offset in ((0, 0), (3, 1)):
        stream = strided(r, pad, offset)
        got = sg.linear_bf16(x, w, b, "gelu", stream, save="bf16", out=stream)
        assert torch.equal(got.y, want.y) and torch.equal(got.pre, want.pre)
        assert int(stream.as_strided((T * (O + pad),), (1,)).isnan().sum()) == T * pad
    calls = []
    for seed, (T, I, O) in enumerate(((16384, 1024, 256), (2, 128, 8413))):
        dy, x, w, u = rand(seed, T, O, std=0.1), rand(seed + 1, T, I), rand(seed + 2, O, I, std=O ** -0.5), rand(seed + 3, O, I, std=O ** -0.5)
        a, v = rand(seed + 4, T, O), rand(seed + 5, T, O)
        check_all(sg.linear_bf16_backward(dy, x, w, a, "silu", dbias=True, dweight_dtype=torch.float32), linear_grad_ref(dy, x, w, a, "silu"))
        calls.append(lambda dy=dy, x=x, w=w, u=u, a=a, v=v: sg.gated_bf16_backward(dy, x, w, u, a, v, "gelu", h=True))
        check_all(calls[-1](), gated_grad_ref(dy, x, w, u, a, v, "gelu"))
    want = [call() for call in calls]
    graphs, got, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for call in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(call())
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for p, q in zip(want, got):
        assert all(torch.equal(m, n) for m, n in zip(p, q))
    done()


@pytest.mark.parametrize("kernel", [("AUTO", 0, 0), ("LINEAR_PAIR", 256, 1), ("LINEAR_PAIR", 128, 0), ("LINEAR_PAIR", 128, 4), ("LINEAR_SHORT", 64, 1)], ids=str)
def test_fp32_values_of_any_length(force, kernel):
    """FP32 outputs and the scales of 8-bit values do not drift with K.  The tensor cores round each of the 4 steps of a K tile
    towards zero: half a unit of the last place on average, which is 0.72 u of a value (u 2^-24; its mean over a binade), of
    partial sums that are half of the whole one on average, so 4 * 0.72 / 2 = 1.44 u per K tile of an accumulator at most.
    Measured it is 1.02 u, 6.1e-8, which is what the kernel's rule goes by: accumulators of n_i K tiles, whose sums are
    independent and go by the roots of their lengths, are together off by 6.1e-8 sqrt(sum(n_i^3) / sum(n_i)) of the whole sum,
    and the rule keeps the root at 13.  This test holds it to that, with u for the FP32 sums and a tenth of room.  (The guaranteed
    bound, (K + 2) u sum|a b|, is the other tests'.)"""
    import torch
    force(*kernel)
    tol = 1.1 * (13 * 6.1e-8 + 2.0 ** -24)  # 9.4e-7
    worst = []
    for kt in (1, 8, 12, 13, 14, 15, 16, 17, 20, 24, 32, 47, 49, 64, 100, 128, 200):
        T, I, O = 300, 64 * kt, 256
        x, w, u = rand(kt, T, I), rand(kt + 1, O, I, std=I ** -0.5), rand(kt + 2, O, I, std=I ** -0.5)
        pre = x.double() @ w.double().T
        scale = pre.abs().view(T, -1, 128).amax(2) / 448
        off = lambda got, want: float((got.double() - want).norm() / want.norm())  # noqa: E731
        worst.append(max(off(sg.linear_bf16(x, w, out_dtype=torch.float32).y, pre), off(sg.linear_bf16(x, w, save="fp8").pre.scale, scale),
                         off(sg.gated_bf16(x, w, u, save="fp8").gate.scale, scale)))
    assert max(worst) <= tol, worst
    done()


def test_empty():
    """No tokens, no inputs, no outputs: empty results and sums of nothing."""
    import torch
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    b, r = rand(1, 1, 70)[0], rand(2, 40, 70)
    for T in (1, 40, 300):
        rr = rand(2, T, 70)
        got = sg.linear_bf16(e(T, 0), e(70, 0), b, "silu", rr, save="fp8")  # the bias's activation, and the residual
        ref = linear_ref(torch.zeros(T, 1, device="cuda"), torch.zeros(70, 1, device="cuda"), b, "silu", rr)
        check_all(got, ref, ["y"])
        check_kept(got.pre, *ref["pre"])
        assert bool((sg.gated_bf16(e(T, 0), e(70, 0), e(70, 0)).h == 0).all())
    assert sg.linear_bf16(e(0, 64), e(70, 64), b).y.shape == (0, 70) and sg.gated_bf16(e(5, 64), e(0, 64), e(0, 64)).h.shape == (5, 0)
    g = sg.linear_bf16_backward(e(0, 70), e(0, 64), rand(1, 70, 64), dbias=True)
    assert g.dx.shape == (0, 64) and bool((g.dweight == 0).all()) and bool((g.dbias == 0).all())
    g = sg.linear_bf16_backward(e(40, 0), rand(1, 40, 64), e(0, 64), dbias=True)
    assert g.dweight.shape == (0, 64) and bool((g.dx == 0).all()) and g.dbias.shape == (0,)
    g = sg.linear_bf16_backward(r, e(40, 0), e(70, 0), dbias=True)
    assert g.dx.shape == (40, 0) and g.dweight.shape == (70, 0)
    close(g.dbias, r.double().sum(0), 56 * 2.0 ** -24 * r.double().abs().sum(0))
    g = sg.gated_bf16_backward(e(0, 70), e(0, 64), rand(1, 70, 64), rand(2, 70, 64), e(0, 70), e(0, 70), h=True)
    assert bool((g.dgate == 0).all()) and bool((g.dup == 0).all()) and g.dx.shape == (0, 64) and g.h.shape == (0, 70)
    g = sg.gated_bf16_backward(e(40, 0), rand(1, 40, 64), e(0, 64), e(0, 64), e(40, 0), e(40, 0), h=True)
    assert bool((g.dx == 0).all()) and g.dup.shape == (0, 64) and g.h.shape == (40, 0)
    g = sg.gated_bf16_backward(r, e(40, 0), e(70, 0), e(70, 0), r, r, None, h=True)
    close(g.h, r.double() ** 2, rounded(r.double() ** 2, 4 * 2.0 ** -24 * r.double() ** 2, torch.bfloat16))
    done()


def test_only_what_is_wanted(force):
    """Each output alone: the same values where the kernel is the same, None for the others."""
    import torch
    T, I, O = 70, 200, 136
    force("LINEAR_PAIR", 128)
    dy, x, w, u, a, b = rand(1, T, O), rand(2, T, I), rand(3, O, I), rand(4, O, I), rand(5, T, O), rand(6, T, O)
    full = sg.linear_bf16_backward(dy, x, w, a, "gelu", dbias=True)
    only = [sg.linear_bf16_backward(dy, None, w, a, "gelu", dweight=False), sg.linear_bf16_backward(dy, x, None, a, "gelu", dx=False),
            sg.linear_bf16_backward(dy, None, None, a, "gelu", dx=False, dweight=False, dbias=True)]
    assert only[0].dweight is None and only[0].dbias is None and torch.equal(only[0].dx, full.dx)
    assert only[1].dx is None and torch.equal(only[1].dweight, full.dweight)
    assert only[2].dx is None and only[2].dweight is None and torch.equal(only[2].dbias, full.dbias)
    full = sg.gated_bf16_backward(dy, x, w, u, a, b, h=True)
    one = sg.gated_bf16_backward(dy, None, w, u, a, b, dweights=False)
    assert torch.equal(one.dx, full.dx) and one[1:] == (None, None, None)
    one = sg.gated_bf16_backward(dy, x, None, None, a, b, dx=False)
    assert torch.equal(one.dgate, full.dgate) and torch.equal(one.dup, full.dup) and one.dx is None and one.h is None
    one = sg.gated_bf16_backward(dy, None, None, None, a, b, dx=False, dweights=False, h=True)
    assert torch.equal(one.h, full.h) and one[:3] == (None, None, None)
    force()
    check_all(sg.gated_bf16_backward(dy, None, w, u, a, b, dweights=False), gated_grad_ref(dy, x, w, u, a, b, "silu"), ["dx"])
    done()


@pytest.mark.parametrize("kernel", [("LINEAR_SHORT", 32, 2), ("LINEAR_PAIR", 256, 0)], ids=str)
def test_non_finite_values(force, kernel):
    """A NaN or an infinity reaches the elements whose sums it enters and no others, a group's scale is that of its finite
    values, and codes have NaN in their places."""
    import torch
    force(*kernel)
    T, I, O = 40, 300, 256
    x, w = rand(1, T, I), rand(2, O, I, std=I ** -0.5)
    x[3, 5], x[7, 9], w[130, 2] = float("nan"), float("inf"), float("inf")
    got = sg.linear_bf16(x, w, None, None, save="fp8")
    want = x.double() @ w.double().T
    odd = ~want.isfinite()
    assert torch.equal(got.y.isnan(), want.isnan()) and torch.equal(got.y.isinf(), want.isinf())
    assert torch.equal(got.pre.data.float().isnan(), odd)
    finite = torch.where(odd, 0.0, want)
    s = (finite.abs().view(T, 2, 128).amax(2) / 448).clamp_min(2.0 ** -126)
    assert float(((got.pre.scale.double() - s) / s).abs().max()) < 1e-5
    h = sg.gated_bf16(x, w, rand(3, O, I)).h
    assert bool(h[3].isnan().all()) and bool(h[8:, :130].isfinite().all())
    done()


@pytest.mark.parametrize("activation", ACTS[1:])
def test_activations_over_their_range(activation):
    """Every finite BF16 value through the activation (as a bias on a product of nothing), and its derivative there."""
    import torch
    a = torch.arange(0, 65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    a = a[a.isfinite()]
    n = a.numel()
    e = torch.empty
    f, df = (v.float() for v in _act64(a.double(), activation))
    y = sg.linear_bf16(e(1, 0, dtype=a.dtype, device="cuda"), e(n, 0, dtype=a.dtype, device="cuda"), a, activation, out_dtype=torch.float32).y[0]
    small = a.abs() < 80  # beyond, FP32's exp() is 0 or infinite: f is a, or 0 to 2^-100
    tol = 16 * 2.0 ** -24 * a.double().abs() + 2.0 ** -100
    close(y, f.double(), tol)
    assert bool((y[~small & (a > 0)] == a[~small & (a > 0)].float()).all())
    one = torch.ones(1, n, dtype=a.dtype, device="cuda")
    d = sg.linear_bf16_backward(one, None, None, a[None], activation, dx=False, dweight=False, dbias=True).dbias
    close(d, df.double(), 32 * 2.0 ** -24 * (1 + a.double().abs().clamp_max(80)))
    # infinities: the derivative's limits
    inf = torch.tensor([[float("inf"), float("-inf")]], dtype=a.dtype, device="cuda")
    d = sg.linear_bf16_backward(torch.ones_like(inf), None, None, inf, activation, dx=False, dweight=False, dbias=True).dbias
    assert d.tolist() == [1.0, 0.0]
    done()


def _act64(a, activation):
    import torch
    from linear_util import act
    f, df = act(a, activation)
    return torch.nan_to_num(f, nan=0.0), torch.where(a.abs() > 80, (a > 0).double(), df)


def test_gradients_against_differences():
    """dX, dW and dbias of a layer and dX, dG, dU of a gated block against central differences of the forward pass in 64 bits
    along random directions: the backward pass is that of this forward pass."""
    import torch
    from linear_util import act
    T, I, O = 24, 40, 56
    x, w, u, b = (rand(i, *s).double() for i, s in ((1, (T, I)), (2, (O, I)), (3, (O, I)), (4, (1, O))))
    w, u, dy = w * 0.2, u * 0.2, rand(5, T, O)
    step = 1e-5
    for activation in ACTS[2:]:
        layer = lambda x, w, b: (act(x @ w.T + b, activation)[0] * dy.double()).sum()  # noqa: E731
        block = lambda x, w, u: (act(x @ w.T, activation)[0] * (x @ u.T) * dy.double()).sum()  # noqa: E731
        xb, wb, ub = x.bfloat16(), w.bfloat16(), u.bfloat16()
        x_, w_, u_ = xb.double(), wb.double(), ub.double()
        pre = (x_ @ w_.T + b).bfloat16()
        g = sg.linear_bf16_backward(dy, xb, wb, pre, activation, dbias=True)
        k = sg.gated_bf16_backward(dy, xb, wb, ub, (x_ @ w_.T).bfloat16(), (x_ @ u_.T).bfloat16(), activation)
        for f, at, grads in ((layer, [x_, w_, b], [g.dx, g.dweight, g.dbias[None]]), (block, [x_, w_, u_], [k.dx, k.dgate, k.dup])):
            for i, grad in enumerate(grads):
                v = torch.sign(grad.double())  # the direction in which nothing cancels
                lo, hi = ([p - step * v if j == i else p for j, p in enumerate(at)], [p + step * v if j == i else p for j, p in enumerate(at)])
                slope = float((f(*hi) - f(*lo)) / (2 * step))
                along = float((grad.double() * v).sum())
                # each factor was rounded to BF16 a few times: 2^-8 each of a sum of positive terms; the rounded values
                # before the activation change its derivative by 2^-8 |a| |f''| (at most about 1) too
                assert abs(along - slope) <= 8 * 2.0 ** -8 * abs(slope), (activation, i)
    done()


def test_a_block_as_it_is_trained():
    """The operators together: a gated block with its second layer, forward, 8-bit values, backward, against the same in
    64 bits from what the forward pass kept; the norm's 8-bit output is the layer's input."""
    import torch
    T, I, O = 300, 256, 384
    x0, gain = rand(1, T, I), rand(2, 1, I)[0]
    gate, up, down = rand(3, O, I, std=I ** -0.5), rand(4, O, I, std=I ** -0.5), rand(5, I, O, std=O ** -0.5)
    n = sg.rmsnorm_fp8(x0, gain, y=True)
    mid = sg.gated_bf16(n.y, gate, up, save="fp8")
    y = sg.linear_bf16(mid.h, down, residual=x0).y
    check_all(mid, gated_ref(n.y, gate, up, "silu"), ["h"])
    ref = linear_ref(mid.h, down, None, None, x0)["y"]
    close(y, ref[0], rounded(*ref, y.dtype))
    dy = rand(6, T, I, std=0.1)
    again = sg.gated_bf16_backward(dy.new_zeros(T, O), None, gate, up, mid.gate, mid.up, dx=False, dweights=False, h=True).h
    last = sg.linear_bf16_backward(dy, again, down)
    check_all(last, linear_grad_ref(dy, again, down, None, None), ["dx", "dweight"])
    got = sg.gated_bf16_backward(last.dx, n.q, gate, up, mid.gate, mid.up, h=True)
    check_all(got, gated_grad_ref(last.dx, n.q, gate, up, mid.gate, mid.up, "silu"))
    assert torch.equal(got.h, again)
    dx0, dgain = sg.rmsnorm_fp8_backward(got.dx, x0, gain, n.rstd, dy)
    assert bool(dx0.isfinite().all()) and bool(dgain.isfinite().all())
    done()


def test_graphs_and_streams():
    """Captured calls replayed on new values, two graphs in flight on two streams, and a call on a stream of its own give
    the eager results."""
    import torch
    T, I, O = 130, 520, 264
    x, w, u = rand(1, T, I), rand(2, O, I, std=0.05), rand(3, O, I, std=0.05)
    dh = rand(4, T, O)
    odd = strided(x, 3)  # (copied in the workspace)

    def step(x, odd):
        f = sg.gated_bf16(x, w, u, save="fp8")
        g = sg.gated_bf16_backward(dh, odd, w, u, f.gate, f.up, h=True)
        e = sg.linear_bf16_backward(dh, odd, w, g.h, "gelu", dbias=True)
        return f.h, *g, *e, sg.linear_bf16(odd, w, None, "relu", g.h).y
    step(x, odd)
    graphs, outs, ins = [], [], []
    for k in range(2):
        a, b = x.clone(), strided(x, 3)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out = step(a, b)
        graphs.append(graph), outs.append(out), ins.append((a, b))
    wants = []
    for k in range(2):
        v = rand(10 + k, T, I)
        ins[k][0].copy_(v), ins[k][1].copy_(v)
        wants.append(step(v, strided(v, 3)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        assert all(torch.equal(p, q) for p, q in zip(out, want))
    v = rand(10, T, I)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = sg.linear_bf16(v, w, stream=s).y
    s.synchronize()
    assert torch.equal(y, sg.linear_bf16(v, w).y)
    done()


def test_results_do_not_depend_on_the_run():
    import torch
    for T, I, O in ((1, 4096, 512), (64, 2048, 520), (1000, 1300, 700)):
        x, w, dy, a = rand(1, T, I), rand(2, O, I), rand(3, T, O), rand(4, T, O)
        first = (*sg.linear_bf16(x, w, None, "gelu", save="bf16"), *sg.linear_bf16_backward(dy, x, w, a, "gelu", dbias=True))
        for _ in range(5):
            again = (*sg.linear_bf16(x, w, None, "gelu", save="bf16"), *sg.linear_bf16_backward(dy, x, w, a, "gelu", dbias=True))
            assert all(torch.equal(p, q) for p, q in zip(first, again))
    done()


def test_beyond_31_bits():
    """Outputs of more than 2^31 elements, and rows more than 2^31 elements apart from the first: their ends are right."""
    import torch
    T, I, O = 131200, 64, 16640
    x, w = rand(1, T, I), rand(2, O, I)
    y = sg.linear_bf16(x, w, None, "relu").y
    rows = torch.tensor([0, 1, 70000, T - 257, T - 1], device="cuda")
    ref = linear_ref(x[rows], w, None, "relu", None)["y"]
    close(y[rows], ref[0], rounded(*ref, y.dtype))
    a = y  # as values that were kept, and as a gradient
    g = sg.linear_bf16_backward(y, x, w, a, "gelu", dbias=True)
    pre, f = y[rows].double(), linear_grad_ref(y[rows], x[rows], w, a[rows], "gelu")
    close(g.dx[rows], f["dx"][0], rounded(*f["dx"], g.dx.dtype))
    del pre, g
    k = sg.gated_bf16(x, w, w, "relu", save="fp8")
    ref = gated_ref(x[rows], w, w, "relu")
    close(k.h[rows], ref["h"][0], rounded(*ref["h"], k.h.dtype))
    m = sg.Fp8Matrix(k.gate.data[T - 257:], k.gate.scale[T - 257:])
    close(values(m)[-1:], ref["gate"][0][-1:], ref["gate"][1][-1:] + (2.0 ** -4 + 1e-5) * ref["gate"][0][-1:].abs() + 2.0 ** -10 * m.scale[-1].max().double())
    done()
