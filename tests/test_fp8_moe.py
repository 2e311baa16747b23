"""The mixture-of-experts layer for a few tokens (sgemm_fp8_moe) against the formula in 64 bits.

Tolerance.  A dot product of n FP32 terms is within (n + 2) u of the sum of magnitudes (u = 2^-24); the inner
values are within 2^-9.8 of the largest of their 64 columns (two 8-bit terms), and the second product carries
both errors through |W2|; BF16 output adds 2^-8 of the result."""
import numpy as np
import pytest

import sgemm_row_major_gb300 as sg
from fp8_util import U, code_values, spread

FAKE = 1 << 20


def layer(T, E, H, I, seed, pad=0):
    import torch
    rng = np.random.default_rng(seed)
    vals = code_values("e4m3")
    usable = np.flatnonzero((np.abs(vals) <= 16) & (np.abs(vals) >= 2.0 ** -4))

    def make(shape, block, amp):
        rows, cols = shape[-2:]
        codes = rng.choice(usable, shape).astype(np.uint8)
        scale = (rng.uniform(0.5, 1.5, shape[:-2] + (-(-rows // block[0]), -(-cols // block[1]))) * amp).astype(np.float32)
        buf = np.full(shape[:-1] + (cols + pad,), 0x7F, np.uint8)
        buf[..., :cols] = codes
        t = torch.from_numpy(buf).cuda()[..., :cols].view(torch.float8_e4m3fn)
        ref = vals[codes] * (spread(scale, block, (rows, cols)) if len(shape) == 2
                             else np.stack([spread(s, block, (rows, cols)) for s in scale]))
        return t, torch.from_numpy(scale).cuda(), ref
    xd, xs, x = make((T, H), (1, 128), 0.2)
    ws = [make((E, *s), (128, 128), 0.25 / s[1] ** 0.5) for s in ((I, H), (I, H), (H, I))]
    logits = rng.standard_normal((T, E)).astype(np.float32)
    return sg.Fp8Matrix(xd, xs), x, logits, [(w[0], w[1]) for w in ws], [w[2] for w in ws]


def reference(x, logits, k, ws, renormalize):
    """(y, tolerance in FP32)."""
    T, E = logits.shape
    H, I = ws[2].shape[1:]
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        lg = logits[t].astype(np.float64)
        if np.isnan(lg).any() or np.isposinf(lg).any():
            y[t] = np.nan
            continue
        order = [e for e in np.argsort(-lg, kind="stable")[:k] if np.isfinite(lg[e])]
        if not order:
            continue
        p = np.exp(lg - lg.max())
        p /= p[order].sum() if renormalize else p.sum()
        for e in order:
            g, u = ws[0][e] @ x[t], ws[1][e] @ x[t]
            mg, mu = np.abs(ws[0][e]) @ np.abs(x[t]), np.abs(ws[1][e]) @ np.abs(x[t])
            s = 1 / (1 + np.exp(-g))
            h = g * s * u
            # |d silu| <= 1.1 |dg|
            dh = (H + 4) * U * (1.1 * mg * np.abs(u) + np.abs(g * s) * mu) + 8 * U * np.abs(h)
            big = np.pad(np.abs(h), (0, -I % 64)).reshape(-1, 64).max(1).repeat(64)[:I]
            dh += 2.0 ** -9.8 * big * (1 + 2.0 ** -6)
            y[t] += p[e] * (ws[2][e] @ h)
            tol[t] += p[e] * (np.abs(ws[2][e]) @ (dh + (2 * I + E + 8) * U * np.abs(h)))
    return y, tol


def check(T, E, k, H, I, seed, renormalize=True, bf16=True, logits=None, pad=0):
    import torch
    x, xr, lg, ws, wr = layer(T, E, H, I, seed, pad)
    if logits is not None:
        lg = logits(lg)
    got = sg.moe_fp8(x, torch.from_numpy(lg).cuda(), k, *ws, renormalize=renormalize,
                     out_dtype=torch.bfloat16 if bf16 else torch.float32)
    assert sg.sgemm_sync_status(torch.cuda.current_stream()) == 0
    y, tol = reference(xr, lg, k, wr, renormalize)
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(y))
    fine = ~np.isnan(y)
    err = np.abs(g - y)[fine]
    lim = (tol + (2.0 ** -8 * (np.abs(y) + tol) if bf16 else U * np.abs(y)))[fine]
    assert np.all(err <= lim), (float((err / np.maximum(lim, 1e-300)).max()), np.argwhere(np.abs(g - y) > tol + 2.0 ** -8 * np.abs(y))[:4])
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 16, 16), (1, 8, 2, 128, 128), (1, 64, 8, 512, 256), (2, 5, 5, 144, 208), (7, 16, 3, 400, 336),
                                       (16, 8, 2, 256, 1040), (17, 40, 6, 656, 64), (33, 12, 4, 384, 192), (64, 128, 8, 256, 128),
                                       (64, 2, 2, 1040, 144), (5, 1000, 16, 128, 128), (33, 26, 4, 2048, 1024), (3, 26, 4, 2048, 1024)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_against_the_formula(T, E, k, H, I, renormalize):
    check(T, E, k, H, I, T + E + k, renormalize, bf16=renormalize)


@pytest.mark.gpu
@pytest.mark.parametrize("inner", [3, 70, 133, 200])
@pytest.mark.parametrize("I", [208, 256])
def test_nan_inner_value_under_a_zero_scale(inner, I):
    """A NaN inner value times weights whose scale is 0 is NaN, in whichever half of a group of 128 it lies."""
    import torch
    x, xr, lg, ws, wr = layer(3, 4, 256, I, 12)
    ws[0][0].view(torch.uint8)[:2, inner] = 0x7F
    wr[0][:2, inner] = np.nan
    ws[2][1][..., inner // 128] = 0.0
    wr[2][..., 128 * (inner // 128): 128 * (inner // 128) + 128] *= 0.0
    lg[0], lg[1] = [9, 8, 1, 2], [1, 2, 9, 8]
    got = sg.moe_fp8(x, torch.from_numpy(lg).cuda(), 2, *ws, out_dtype=torch.float32).cpu().numpy()
    y, tol = reference(xr, lg, 2, wr, True)
    assert np.isnan(y[0]).all() and np.isfinite(y[1]).all()
    assert np.array_equal(np.isnan(got), np.isnan(y)), (np.isnan(got).sum(1), np.isnan(y).sum(1))
    assert np.all(np.abs(got[1] - y[1]) <= tol[1] + U * np.abs(y[1]))


def largest_codes(data, scale, ref, block):
    """Every code replaced by the largest one of the same sign."""
    import torch
    data.view(torch.uint8).bitwise_or_(0x7E).bitwise_and_(0xFE)
    s = scale.double().cpu().numpy().reshape(-1, *scale.shape[-2:])
    ref[:] = np.copysign(448.0 * np.stack([spread(m, block, ref.shape[-2:]) for m in s]).reshape(ref.shape), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,H,I", [(3, 6, 2, 256, 256), (40, 6, 3, 256, 160)])
def test_each_scale_may_be_extreme(T, E, k, H, I):
    """Scales far from 1 on either side of a product whose value is ordinary: x against gate and up, and inner values
    of 2^118 against down.  A group's sum times one of them alone would be beyond FP32."""
    import torch
    big, small = 2.0 ** 118, 2.0 ** -118
    for inner_big in (False, True):
        x, xr, lg, ws, wr = layer(T, E, H, I, 11)
        if inner_big:
            largest_codes(*ws[2], wr[2], (128, 128))
            ws[1][1].mul_(big)
            wr[1] *= big
            ws[2][1].mul_(small)
            wr[2] *= small
        else:
            largest_codes(x.data, x.scale, xr, (1, 128))
            for m, m_ref, f in ((x.scale, xr, big), (ws[0][1], wr[0], small), (ws[1][1], wr[1], small)):
                m[..., 0].mul_(f)
                m_ref[..., :128] *= f
                m[..., 1].mul_(1 / f)
                m_ref[..., 128:] *= 1 / f
        got = sg.moe_fp8(x, torch.from_numpy(lg).cuda(), k, *ws, out_dtype=torch.float32)
        y, tol = reference(xr, lg, k, wr, True)
        assert np.isfinite(y).all()
        err = np.abs(got.double().cpu().numpy() - y)
        assert np.all(err <= tol + U * np.abs(y)), (inner_big, float(np.nanmax(err / tol)), int((~np.isfinite(err)).sum()))


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,H,I", [(16, 256, 16, 2048, 784), (20, 100, 8, 2048, 784), (40, 40, 4, 2048, 784),   # one kernel after the other
                                       (16, 128, 16, 2048, 784), (20, 60, 8, 2048, 784), (40, 24, 4, 2048, 784)])  # beside each other
def test_both_launch_forms(T, E, k, H, I):
    """Layers with many weights per SM, in which the kernels run one after the other, and with fewer."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(E)

    def stack(rows, cols):
        codes = torch.randint(0x18, 0x58, (E, rows, cols), generator=g, device="cuda", dtype=torch.uint8)  # 2^-4 .. 15
        codes |= torch.randint(0, 2, (E, rows, cols), generator=g, device="cuda", dtype=torch.uint8) << 7
        return codes.view(torch.float8_e4m3fn), (torch.rand(E, -(-rows // 128), -(-cols // 128), generator=g, device="cuda") + 0.5) * (0.25 / cols ** 0.5)

    def real(w, e):
        return w[0][e].double() * w[1][e].double().repeat_interleave(128, 0)[: w[0].shape[1]].repeat_interleave(128, 1)[:, : w[0].shape[2]]
    x = sg.quantize_fp8(torch.randn(T, H, generator=g, device="cuda"))
    xr = x.data.double() * x.scale.double().repeat_interleave(128, 1)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ws = [stack(I, H), stack(I, H), stack(H, I)]
    got = sg.moe_fp8(x, logits, k, *ws, out_dtype=torch.float32)
    assert torch.equal(sg.moe_fp8(x, logits, k, *ws, out_dtype=torch.float32), got)
    assert sg.sgemm_sync_status(torch.cuda.current_stream()) == 0
    p, at = logits.double().softmax(1).topk(k, 1)
    p /= p.sum(1, keepdim=True)
    y, tol = torch.zeros(2, T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (at == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        w1, w3, w2 = (real(w, e) for w in ws)
        gate, up, mg, mu = xr[t] @ w1.T, xr[t] @ w3.T, xr[t].abs() @ w1.abs().T, xr[t].abs() @ w3.abs().T
        s = torch.sigmoid(gate)
        h = gate * s * up
        big = torch.nn.functional.pad(h.abs(), (0, -I % 64)).view(len(t), -1, 64).amax(2).repeat_interleave(64, 1)[:, :I]
        dh = (H + 4) * U * (1.1 * mg * up.abs() + (gate * s).abs() * mu) + 8 * U * h.abs() + 2.0 ** -9.8 * big * (1 + 2.0 ** -6)
        c = p[t, j][:, None]
        y[t] += c * (h @ w2.T)
        tol[t] += c * ((dh + (2 * I + E + 8) * U * h.abs()) @ w2.abs().T)
    err = (got.double() - y).abs()
    assert bool((err <= tol + U * y.abs()).all()), float((err / tol).max())


@pytest.mark.gpu
def test_every_token_to_one_expert():
    """All tokens on the same experts (a full tile of columns), and each token on an expert of its own."""
    def same(lg):
        lg[:, 3] = 9.0
        lg[:, 1] = 8.0
        return lg
    check(64, 6, 2, 256, 320, 1, logits=same)

    def own(lg):
        lg[:] = -5.0
        lg[np.arange(40), np.arange(40)] = 5.0
        return lg
    check(40, 40, 1, 256, 320, 2, logits=own)


@pytest.mark.gpu
def test_masked_and_tied_logits():
    """-Inf is never chosen, a row of them gives zeros; NaN and +Inf give NaN rows; ties go to the lowest index (-0 equals 0)."""
    def masked(lg):
        lg[0] = -np.inf
        lg[1, 2:] = -np.inf
        lg[2, 5] = np.nan
        lg[3, 0] = np.inf
        lg[4] = 1.25
        lg[5, ::2], lg[5, 1::2] = 0.0, -0.0
        lg[6, 3] = np.float32(-3e38)
        lg[6, 4:] = -np.inf
        return lg
    for renormalize in (True, False):
        got = check(9, 12, 4, 144, 160, 3, renormalize, logits=masked)
        assert bool((got[0] == 0).all())


@pytest.mark.gpu
def test_row_strides_and_scale_strides():
    check(3, 6, 2, 144, 160, 4, pad=16)
    import torch
    x, xr, lg, ws, wr = layer(4, 6, 256, 256, 5)
    big = torch.full((4, 300), 0x7F, dtype=torch.uint8, device="cuda")[:, 3:259]  # rows TMA cannot read
    big.copy_(x.data.view(torch.uint8))
    xs = torch.full((4, 7), float("nan"), device="cuda")[:, :2]
    xs.copy_(x.scale)
    wide = torch.full((4, 270), 7.0, device="cuda")
    logits = torch.full((4, 9), float("nan"), device="cuda")[:, :6]
    logits.copy_(torch.from_numpy(lg))
    want = sg.moe_fp8(x, torch.from_numpy(lg).cuda(), 2, *ws, out_dtype=torch.float32)
    sg.moe_fp8(sg.Fp8Matrix(big.view(torch.float8_e4m3fn), xs), logits, 2, *ws, out=wide[:, :256])
    assert torch.equal(wide[:, :256], want) and bool((wide[:, 256:] == 7.0).all())


@pytest.mark.gpu
def test_fused_gate_and_up_rows():
    """Gate and up as the halves of one stored matrix per expert: strides larger than a matrix."""
    import torch
    x, xr, lg, ws, wr = layer(5, 4, 256, 128, 6)
    both = torch.cat([ws[0][0].view(torch.uint8), ws[1][0].view(torch.uint8)], 1).view(torch.float8_e4m3fn)
    scale = torch.cat([ws[0][1], ws[1][1]], 1)
    lg = torch.from_numpy(lg).cuda()
    want = sg.moe_fp8(x, lg, 2, *ws)
    got = sg.moe_fp8(x, lg, 2, (both[:, :128], scale[:, :1]), (both[:, 128:], scale[:, 1:]), ws[2])
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_repeatable_on_streams_and_in_graphs():
    import torch
    x, xr, lg, ws, wr = layer(20, 16, 512, 384, 7)
    lg = torch.from_numpy(lg).cuda()
    want = sg.moe_fp8(x, lg, 4, *ws)
    assert torch.equal(sg.moe_fp8(x, lg, 4, *ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sg.moe_fp8(x, lg, 4, *ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sg.moe_fp8(x, lg, 4, *ws)
    first = want.clone()
    lg.copy_(lg.flip(1).contiguous())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, sg.moe_fp8(x, lg, 4, *ws)) and not torch.equal(got, first)


@pytest.mark.gpu
def test_nothing_to_do():
    import torch
    x, xr, lg, ws, wr = layer(3, 4, 128, 128, 8)
    lg = torch.from_numpy(lg).cuda()
    assert bool((sg.moe_fp8(x, lg, 0, *ws) == 0).all())
    assert sg.moe_fp8(sg.Fp8Matrix(x.data[:0], x.scale[:0]), lg[:0], 2, *ws).shape == (0, 128)


def test_refusals():
    from sgemm_row_major_gb300 import fp8
    lib = fp8._lib()

    def w(rows, cols, **kw):
        a = dict(data=FAKE, ld=cols, stride=rows * cols, scale=FAKE, lds=-(-cols // 128), stride_scale=-(-rows // 128) * -(-cols // 128))
        a.update(kw)
        return fp8.ExpertsStruct(*a.values())

    def x(**kw):
        a = dict(data=FAKE, ld=256, scale=FAKE, lds=2, format=0, block_rows=1, block_cols=128)
        a.update(kw)
        return fp8.MatrixStruct(*a.values())
    ok = [4, 256, 512, 8, 2, x(), FAKE, 8, 1, w(512, 256), w(512, 256), w(256, 512), FAKE, 256, 1, None]
    bad = [(1, -1), (2, -1), (3, -1), (4, -1), (5, 9), (5, -1), (6, None), (6, x(format=1)), (6, x(block_rows=128)), (6, x(ld=255)),
           (6, x(lds=1)), (7, None), (8, 7), (10, None), (13, None), (13, FAKE + 1), (14, 255), (15, 2)]
    for i, (rows, cols) in ((10, (512, 256)), (11, (512, 256)), (12, (256, 512))):
        bad += [(i, w(rows, cols, data=FAKE + 8)), (i, w(rows, cols, ld=cols + 8)), (i, w(rows, cols, stride=rows * cols - 16)),
                (i, w(rows, cols, stride=rows * cols + 8)), (i, w(rows, cols, scale=None)), (i, w(rows, cols, lds=1)),
                (i, w(rows, cols, stride_scale=3)), (i, w(rows, cols, data=None))]
    for index, value in bad:
        args = list(ok)
        args[index - 1] = value
        assert lib.sgemm_fp8_moe(*args) == -index, (index, value)
    for index, value in [(1, 65), (2, 264), (3, 520)]:
        args = list(ok)
        args[index - 1] = value
        args[5] = x(ld=1024, lds=9)
        args[9], args[10], args[11] = (w(args[2], 1024, lds=9), w(args[2], 1024, lds=9), w(args[1], 1024, lds=9))
        args[13] = 1024
        assert lib.sgemm_fp8_moe(*args) == 4, (index, value)  # SGEMM_ERR_UNSUPPORTED
