"""Helpers of the tests on BF16 layers: references in 64 bits and the bounds of what FP32 arithmetic and one rounding may be off.

u = 2^-24.  A sum of K products is at most (K + 2) u sum|a b| off.  An activation's slope is at most 1.13 (GELU near 1.4), and it
is evaluated to 16 u |a| (a few ulp of each function and division; GELU's argument is off by 2 u, which changes Phi by at most
2 (a^2 + 1) u Phi, less than 1 u |a| in all).  Its derivative is evaluated to 32 u (1 + |a|) by the same count.  A value rounded
to BF16 is off by 2^-8 of itself, to E4M3 by 2^-4 (or half of the smallest step, 2^-10, times the scale)."""
from __future__ import annotations

import math

U = 2.0 ** -24
BF = 2.0 ** -8
TINY = 2.0 ** -126
ACTS = (None, "relu", "silu", "gelu", "gelu_tanh")


def act(a, name):
    """(f(a), f'(a)) from the definitions, in a's type."""
    import torch
    if name is None:
        return a, torch.ones_like(a)
    if name == "relu":
        return a.clamp_min(0.0), (a > 0).to(a.dtype)
    if name == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s))
    if name == "gelu":
        c = 0.5 * torch.erfc(-a / math.sqrt(2.0))
        return a * c, c + a * torch.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    s = torch.sigmoid(2 * k * (a + 0.044715 * a ** 3))
    return a * s, s + a * s * (1 - s) * 2 * k * (1 + 3 * 0.044715 * a * a)


def values(k):
    """The numbers of a kept matrix in 64 bits."""
    import torch
    if torch.is_tensor(k):
        return k.double()
    return k.data.double() * k.scale.double().repeat_interleave(128, 1)[:, : k.shape[1]]


def close(got, want, tol, what=""):
    import torch
    assert got.shape == want.shape, what
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        i = int(torch.where(bad, err / tol.clamp_min(1e-300), torch.zeros_like(err)).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} off, worst {got.reshape(-1)[i]} for {want.reshape(-1)[i]}, "
                             f"tolerance {tol.reshape(-1)[i]}")


def rounded(want, tol, dtype):
    """The tolerance with the rounding to the output's type."""
    import torch
    half = BF if dtype == torch.bfloat16 else U
    return tol * (1 + half) + half * want.abs() + TINY


def check_kept(k, want, tol, what=""):
    """What was kept of values `want` that FP32 sums give to `tol`."""
    import torch
    if torch.is_tensor(k):
        close(k, want, rounded(want, tol, torch.bfloat16), what)
        return
    rows, cols = want.shape
    pad = (0, -cols % 128)
    groups = lambda v: torch.nn.functional.pad(v, pad).view(rows, -1, 128).amax(2)  # noqa: E731
    s, t = (groups(want.abs()) / 448).clamp_min(TINY), groups(tol) / 448
    close(k.scale, s, t + 2 * U * s, what + " scales")
    wide = lambda v: v.repeat_interleave(128, 1)[:, :cols]  # noqa: E731
    # the code of the FP32 value over its scale (two roundings), and the scale's own error
    close(values(k), want, tol + (2.0 ** -4 + 8 * U) * want.abs() + 2.0 ** -10 * wide(s) + 2 * wide(t) * 448, what + " codes")


def product(a, b):
    """(a b^T, (K + 2) u |a| |b|^T) of 64-bit matrices."""
    return a @ b.T, (a.shape[1] + 2) * U * (a.abs() @ b.abs().T)


def linear_ref(x, w, bias, activation, residual):
    """{name: (value, tolerance before rounding)} of a layer."""
    pre, tol = product(x.double(), w.double())
    if bias is not None:
        pre, tol = pre + bias.double(), tol + 2 * U * bias.double().abs()
    f = act(pre, activation)[0]
    y, ytol = f, 1.13 * tol + (16 * U * pre.abs() if activation else 0.0)
    if residual is not None:
        y, ytol = y + residual.double(), ytol + U * (f.abs() + residual.double().abs())
    return {"pre": (pre, tol), "y": (y, ytol)}


def gated_ref(x, gate, up, activation):
    (a, ta), (b, tb) = product(x.double(), gate.double()), product(x.double(), up.double())
    f = act(a, activation)[0]
    return {"gate": (a, ta), "up": (b, tb), "h": (f * b, (1.13 * ta + 16 * U * a.abs()) * (b.abs() + tb) + f.abs() * tb + 2 * U * (f * b).abs())}


def linear_grad_ref(dy, x, w, pre, activation):
    """{name: (value, tolerance before rounding)}; dA is rounded to BF16 where there is an activation, 8-bit x always."""
    d, x8 = dy.double(), not hasattr(x, "dtype")
    dt, xt = 0 * d, 0 * values(x)
    if activation:
        a = values(pre)
        df = act(a, activation)[1]
        et = d.abs() * (32 * U * (1 + a.abs()))
        d, dt = d * df, et + BF * (d * df).abs() + TINY
    else:
        et = 0 * d
    xv = values(x)
    if x8:
        xt = BF * xv.abs() + TINY
    tokens, outputs = d.shape
    out = {"dbias": (d.sum(0), (tokens + 16) * U * d.abs().sum(0) + et.sum(0))}
    if w is not None:
        wv = w.double()
        out["dx"] = (d @ wv, ((outputs + 2) * U * (1 + BF) * d.abs() + dt) @ wv.abs())
    out["dweight"] = (d.T @ xv, ((tokens + 2) * U * (1 + BF) ** 2 * d.abs() + dt).T @ (xv.abs() + xt) + d.abs().T @ xt)
    return out


def gated_grad_ref(dh, x, gate, up, a, b, activation):
    g, av, bv = dh.double(), values(a), values(b)
    f, df = act(av, activation)
    da, db = g * bv * df, g * f
    ta = (g * bv).abs() * 32 * U * (1 + av.abs()) + (BF + 4 * U) * da.abs() + TINY
    tb = g.abs() * 16 * U * av.abs() + (BF + 4 * U) * db.abs() + TINY
    xv = values(x)
    xt = 0 * xv if hasattr(x, "dtype") else BF * xv.abs() + TINY
    tokens, outputs = g.shape
    sum_tol = (2 * outputs + 2) * U * (1 + BF)
    grow = (tokens + 2) * U * (1 + BF) ** 2
    return {
        "dx": (da @ gate.double() + db @ up.double(), (sum_tol * da.abs() + ta) @ gate.double().abs() + (sum_tol * db.abs() + tb) @ up.double().abs()),
        "dgate": (da.T @ xv, (grow * da.abs() + ta).T @ (xv.abs() + xt) + da.abs().T @ xt),
        "dup": (db.T @ xv, (grow * db.abs() + tb).T @ (xv.abs() + xt) + db.abs().T @ xt),
        "h": (f * bv, 16 * U * (av * bv).abs() + 2 * U * (f * bv).abs()),
    }


def check_all(got, ref, names=None):
    for name in names or ref:
        value, tol = ref[name]
        out = getattr(got, name)
        close(out, value, rounded(value, tol, out.dtype), name)
