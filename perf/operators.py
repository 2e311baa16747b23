"""The 8-bit operators of libsgemm as cases that can be timed and compared.

Each case runs one operator on inputs made from a seed: with ``own`` false in
plain torch operations (32-bit arithmetic whatever the inputs' type, one
rounding at the end), with ``own`` true through the calls a user of
``sgemm_row_major_gb300`` makes.  ``exact`` gives the same outputs from the
operator's definition in 64 bits.

Operators:

* ``product``   C = alpha op(A) op(B) + beta C on 8-bit matrices with a scale per block of 128
* ``quantize``  8-bit codes and scales of a matrix, in groups of 1x128, 128x1 or 128x128 elements
* ``norm``      h = x + r, root-mean-square norm of h, 8-bit output with scales
* ``norm_grad`` its backward pass
* ``experts``   a mixture-of-experts layer for a few tokens on 8-bit weights
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
F8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TYPE_BYTES = {"f32": 4, "bf16": 2}
GROUPS = {"row": (1, 128), "col": (128, 1), "block": (128, 128)}
TINY = 2.0 ** -126  # the smallest scale


def listed():
    return [
        # one token through one weight matrix: the call of every decoding step, all latency and weight bytes
        product("product 1x4096x4096", 1, 4096, 4096, "NT", out="bf16"),
        # a batch of 64 decoding sequences through a wide layer (a fully connected shape of the library's own benchmark)
        product("product 64x4096x16384", 64, 4096, 16384, "NT", out="f32"),
        # no size a multiple of anything, added to what C holds: the ragged shape of the library's own benchmark
        product("product 4097x3001x2053", 4097, 3001, 2053, "NT", out="f32", alpha=1.5, beta=-0.5),
        # a prompt or training batch through a square layer: the largest call
        product("product 8192x8192x8192", 8192, 8192, 8192, "NT", out="bf16"),
        # a weight gradient: the tokens are summed over, both operands in column groups, added to the gradient so far
        product("weight gradient 4096x4096x8192", 4096, 4096, 8192, "TN", group_a="col", group_b="col", out="f32", beta=1.0),
        # a weight matrix on its way into 8 bits, once per training step
        quantize("quantize 4096x4096 blocks", 4096, 4096, "f32", "block"),
        # the outgoing gradient of a layer, grouped along the tokens for the weight gradient
        quantize("quantize 16384x4096 columns", 16384, 4096, "bf16", "col", fmt="e5m2"),
        # one token's norm between two layers of a decoding step
        norm("norm 1x4096", 1, 4096, "bf16"),
        # a prompt's norm
        norm("norm 16384x4096", 16384, 4096, "bf16"),
        # the norm's gradients in a training step
        dict(norm("norm gradient 8192x4096", 8192, 4096, "bf16"), op="norm_grad"),
        # one token through its 8 experts
        experts("experts 1 token", 1, 64, 8, 2048, 1024),
        # 32 decoding sequences: nearly every expert is hit, each by a few tokens
        experts("experts 32 tokens", 32, 64, 8, 2048, 1024),
    ]


def product(name, M, N, K, ops, group_a="row", group_b="block", fmt_a="e4m3", fmt_b="e4m3", out="f32", alpha=1.0, beta=0.0, packed=False):
    return {"name": name, "op": "product", "M": M, "N": N, "K": K, "ops": ops, "group_a": group_a, "group_b": group_b, "fmt_a": fmt_a, "fmt_b": fmt_b,
            "out": out, "alpha": alpha, "beta": beta, "packed": packed}


def quantize(name, rows, cols, type_, group, fmt="e4m3"):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "type": type_, "group": group, "fmt": fmt}


def norm(name, rows, cols, type_, residual=True):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "type": type_, "residual": residual}


def experts(name, tokens, experts_, top_k, hidden, inner, renormalize=True):
    return {"name": name, "op": "experts", "tokens": tokens, "experts": experts_, "top_k": top_k, "hidden": hidden, "inner": inner, "renormalize": renormalize}


# ------------------------------------------------------------------ drawn cases

LEFT_OUT = (3072,)  # a size that belongs to others' benchmarks


def between(rng, low, high, step=1):
    """A multiple of `step`, spread over the logarithm of [low, high]; one in three is a power of two or the end of the range."""
    if rng.random() < 0.33:
        powers = [2 ** k for k in range(15) if low <= 2 ** k <= high and 2 ** k % step == 0]
        return rng.choice(powers + [high // step * step])
    n = max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))) // step * step)
    return n + step if n in LEFT_OUT else n


def draw(rng):
    op = rng.choice(["product", "product", "product", "quantize", "norm", "norm_grad", "experts"])
    if op == "product":
        while True:
            M, N, K = between(rng, 1, 16384), between(rng, 128, 8192), between(rng, 128, 16384)
            if M * N * K <= 8192 ** 3:
                break
        # the forward product, the gradient of the inputs (the weights as stored), the gradient of the weights
        ops, group_a, group_b, fmt_a = rng.choice([("NT", "row", "block", "e4m3"), ("NN", "row", "block", "e5m2"), ("TN", "col", "col", "e5m2")])
        c = product("", M, N, K, ops, group_a, group_b, fmt_a, out=rng.choice(["f32", "bf16"]), alpha=rng.choice([1.0, 1.5]), beta=rng.choice([0.0, 0.0, 1.0]),
                    packed=rng.random() < 0.25)
    elif op == "quantize":
        c = quantize("", between(rng, 1, 16384), between(rng, 64, 8192), rng.choice(["f32", "bf16"]), rng.choice(["row", "col", "block"]), rng.choice(["e4m3", "e5m2"]))
    elif op in ("norm", "norm_grad"):
        c = dict(norm("", between(rng, 1, 16384), between(rng, 64, 8192), rng.choice(["f32", "bf16"]), rng.random() < 0.75), op=op)
    else:
        while True:
            T, E, k, H, I = between(rng, 1, 64), between(rng, 8, 128), rng.randint(1, 8), between(rng, 512, 4096, 16), between(rng, 256, 2048, 16)
            if E * H * I <= 3e8 and T * k * H * I <= 1e9:
                break
        c = experts("", T, E, k, H, I, rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def activations(g, rows, cols, std=1.0):
    """Values as they leave a layer: near normal, with a few columns much larger than the rest."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * std
    loud = torch.rand(cols, generator=g, device="cuda") < 0.01
    return x * torch.where(loud, 12.0, 1.0)


def in_groups(x, group):
    """x with rows and columns padded by zeros to whole groups, seen as [row groups, group rows, column groups, group columns]."""
    gr, gc = group
    r, c = x.shape
    pr, pc = -r % gr, -c % gc
    if pr or pc:
        x = torch.nn.functional.pad(x, (0, pc, 0, pr))
    return x.view(x.shape[0] // gr, gr, x.shape[1] // gc, gc)


def spread(s, group, rows, cols):
    """The scale of every element of a rows x cols matrix."""
    gr, gc = group
    return s.repeat_interleave(gr, 0)[:rows].repeat_interleave(gc, 1)[:, :cols]


def codes_of(x, group, fmt, ld=None):
    """8-bit codes of x (row stride ld) and the scales of its groups."""
    top = F8_MAX[fmt]
    v = in_groups(x, group)
    s = (v.abs().amax(dim=(1, 3)) / top).clamp_min(TINY)
    q = (v * (1.0 / s)[:, None, :, None]).clamp(-top, top)
    q = q.reshape(q.shape[0] * q.shape[1], -1)[: x.shape[0], : x.shape[1]].to(F8[fmt])
    ld = ld or x.shape[1]
    data = torch.zeros(x.shape[0], ld, dtype=torch.uint8, device="cuda").view(F8[fmt])
    data.view(torch.uint8)[:, : x.shape[1]] = q.contiguous().view(torch.uint8)
    return data[:, : x.shape[1]], s


def aligned(n):
    return (n + 15) // 16 * 16


def prepare(case, seed):
    g = generator(seed)
    state = {"case": case}
    op = case["op"]
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        ta, tb = case["ops"]
        a = activations(g, *((K, M) if ta == "T" else (M, K)))
        b = torch.randn(*((N, K) if tb == "T" else (K, N)), generator=g, device="cuda") * K ** -0.5
        for key, x in (("a", a), ("b", b)):
            group = GROUPS[case["group_" + key]]
            ld = x.shape[1] if case["packed"] else aligned(x.shape[1])
            state[key], state["s" + key] = codes_of(x, group, case["fmt_" + key], ld)
            state["group_" + key] = group
        state["out"] = TYPES[case["out"]]
        state["c"] = torch.randn(M, N, generator=g, device="cuda").to(state["out"]) if case["beta"] else None
    elif op == "quantize":
        x = activations(g, case["rows"], case["cols"], std=0.02)
        state |= {"x": x.to(TYPES[case["type"]]), "group": GROUPS[case["group"]], "fmt": case["fmt"]}
    elif op in ("norm", "norm_grad"):
        t = TYPES[case["type"]]
        rows, cols = case["rows"], case["cols"]
        state |= {"x": activations(g, rows, cols).to(t), "w": (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(t)}
        state["r"] = activations(g, rows, cols, std=2.0).to(t) if case["residual"] else None
        if op == "norm_grad":  # x stands for the sum that the forward pass stored, r for the gradient that reaches it past the norm
            state["dy"] = (1e-2 * torch.randn(rows, cols, generator=g, device="cuda")).to(t)
            state["rstd"] = (state["x"].float().square().mean(1) + EPS).rsqrt()
            state["r"] = (1e-2 * torch.randn(rows, cols, generator=g, device="cuda")).to(t) if case["residual"] else None
    else:
        T, E, k, H, I = case["tokens"], case["experts"], case["top_k"], case["hidden"], case["inner"]
        state["x"], state["sx"] = codes_of(activations(g, T, H), GROUPS["row"], "e4m3", aligned(H))
        state["logits"] = torch.randn(T, E, generator=g, device="cuda") * 1.5
        for key, rows, cols in (("gate", I, H), ("up", I, H), ("down", H, I)):
            # codes drawn as such: the 8-bit form of normal weights is nearly normal itself
            q = torch.empty(E, rows, cols, dtype=torch.uint8, device="cuda").view(F8["e4m3"])
            for e in range(E):
                q[e] = (torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16) * 100).clamp(-448, 448).to(F8["e4m3"])
            state[key] = q
            state["s_" + key] = torch.rand(E, (rows + 127) // 128, (cols + 127) // 128, generator=g, device="cuda") * (0.02 * cols ** -0.5) + 0.005 * cols ** -0.5
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    return (own_run if own else plain_run)(state)


def own_run(state):
    import sgemm_row_major_gb300 as sg
    case, op = state["case"], state["case"]["op"]
    if op == "product":
        a = sg.Fp8Matrix(state["a"], state["sa"], state["group_a"])
        b = sg.Fp8Matrix(state["b"], state["sb"], state["group_b"])
        ta, tb = case["ops"]
        return sg.matmul_fp8(a, b, state["c"], ta, tb, case["alpha"], case["beta"], out=torch.empty(case["M"], case["N"], dtype=state["out"], device="cuda"))
    if op == "quantize":
        m = sg.quantize_fp8(state["x"], state["group"], state["fmt"])
        return {"codes": m.data, "scale": m.scale}
    if op == "norm":
        out = sg.rmsnorm_fp8(state["x"], state["w"], EPS, state["r"])
        got = {"codes": out.q.data, "scale": out.q.scale, "rstd": out.rstd}
        return got if state["r"] is None else got | {"sum": out.h}
    if op == "norm_grad":
        dx, dw = sg.rmsnorm_fp8_backward(state["dy"], state["x"], state["w"], state["rstd"], state["r"])
        return {"dx": dx, "dw": dw}
    x = sg.Fp8Matrix(state["x"], state["sx"])
    return sg.moe_fp8(x, state["logits"], case["top_k"], (state["gate"], state["s_gate"]), (state["up"], state["s_up"]), (state["down"], state["s_down"]),
                      renormalize=case["renormalize"])


def plain_run(state):
    case, op = state["case"], state["case"]["op"]
    if op == "product":
        a = state["a"].float() * spread(state["sa"], state["group_a"], *state["a"].shape)
        b = state["b"].float() * spread(state["sb"], state["group_b"], *state["b"].shape)
        ta, tb = case["ops"]
        c = (a.T if ta == "T" else a) @ (b.T if tb == "T" else b) * case["alpha"]
        if state["c"] is not None:
            c = c + case["beta"] * state["c"].float()
        return c.to(state["out"])
    if op == "quantize":
        q, s = codes_of(state["x"].float(), state["group"], state["fmt"])
        return {"codes": q, "scale": s}
    if op == "norm":
        h = state["x"].float()
        if state["r"] is not None:
            h = h + state["r"].float()
        rstd = (h.square().mean(1) + EPS).rsqrt()
        q, s = codes_of(h * rstd[:, None] * state["w"].float(), GROUPS["row"], "e4m3")
        got = {"codes": q, "scale": s, "rstd": rstd}
        return got if state["r"] is None else got | {"sum": h.to(state["x"].dtype)}
    if op == "norm_grad":
        dy, h, w, rstd = state["dy"].float(), state["x"].float(), state["w"].float(), state["rstd"][:, None]
        n = h * rstd
        dn = dy * w
        dx = rstd * (dn - n * (dn * n).mean(1, keepdim=True))
        if state["r"] is not None:
            dx = dx + state["r"].float()
        return {"dx": dx.to(state["x"].dtype), "dw": (dy * n).sum(0)}
    # experts: the chosen experts' weights are gathered for every token and choice
    T, k = case["tokens"], case["top_k"]
    at = torch.sort(state["logits"], dim=1, descending=True, stable=True).indices[:, :k]
    p = state["logits"].softmax(1).gather(1, at)
    at = at.reshape(-1)
    if case["renormalize"]:
        p = p / p.sum(1, keepdim=True)
    x = (state["x"].float() * spread(state["sx"], GROUPS["row"], *state["x"].shape)).repeat_interleave(k, 0)[:, :, None]
    gate = torch.bmm(chosen(state["gate"], state["s_gate"], at), x)
    up = torch.bmm(chosen(state["up"], state["s_up"], at), x)
    y = torch.bmm(chosen(state["down"], state["s_down"], at), gate * torch.sigmoid(gate) * up)
    return (y.view(T, k, -1) * p[:, :, None]).sum(1).to(torch.bfloat16)


def chosen(q, s, at):
    """The weights of the experts `at` in 32 bits."""
    rows, cols = q.shape[1:]
    q = q.view(torch.uint8)[at].view(F8["e4m3"]).float()
    return q * s[at].repeat_interleave(128, 1)[:, :rows].repeat_interleave(128, 2)[:, :, :cols]


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """run()'s outputs from the definitions in 64 bits.  Codes are given before their rounding to 8 bits (x over its scale): a
    value next to a tie goes either way, but its distance from the unrounded one is the type's."""
    state = prepare(case, seed)
    op = case["op"]
    if op == "product":
        # sum over the groups of k, each with its own scales
        ta, tb = case["ops"]
        qa, sa = state["a"].double(), state["sa"].double()
        qb, sb = state["b"].double(), state["sb"].double()
        if ta == "T":
            qa, sa = qa.T, sa.T
        if tb == "N":
            qb, sb = qb.T, sb.T
        M, N, K = case["M"], case["N"], case["K"]
        c = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        for g in range((K + 127) // 128):
            ks = slice(128 * g, 128 * g + 128)
            left = qa[:, ks] * (sa[:, g] if sa.shape[0] == M else sa[:, g].repeat_interleave(128)[:M])[:, None]
            right = qb[:, ks] * (sb[:, g] if sb.shape[0] == N else sb[:, g].repeat_interleave(128)[:N])[:, None]
            c.addmm_(left, right.T)
        c *= case["alpha"]
        return c if state["c"] is None else c + case["beta"] * state["c"].double()
    if op == "quantize":
        q, s = unrounded(state["x"].double(), state["group"], state["fmt"])
        return {"codes": q, "scale": s}
    if op == "norm":
        h = state["x"].double() + (state["r"].double() if state["r"] is not None else 0.0)
        rstd = 1.0 / torch.sqrt((h * h).sum(1) / h.shape[1] + EPS)
        q, s = unrounded(torch.einsum("rc,r,c->rc", h, rstd, state["w"].double()), (1, 128), "e4m3")
        return {"codes": q, "scale": s, "rstd": rstd} | ({} if state["r"] is None else {"sum": h})
    if op == "norm_grad":
        # y_i = w_i h_i m^(-1/2), m = mean(h^2) + eps: dy_j/dh_i = w_j m^(-1/2) (delta_ij - h_i h_j / (n m)), with m as rstd has it
        dy, h, w, rstd = state["dy"].double(), state["x"].double(), state["w"].double(), state["rstd"].double()
        inner = torch.einsum("rc,c,rc->r", dy, w, h)
        dx = rstd[:, None] * dy * w - (rstd ** 3 * inner / h.shape[1])[:, None] * h
        if state["r"] is not None:
            dx = dx + state["r"].double()
        return {"dx": dx, "dw": torch.einsum("rc,rc,r->c", dy, h, rstd)}
    # experts, one after the other, each with the tokens that chose it
    logits = state["logits"].double()
    at = torch.argsort(logits, dim=1, descending=True, stable=True)[:, : case["top_k"]]
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    p = e / (e.gather(1, at).sum(1, keepdim=True) if case["renormalize"] else e.sum(1, keepdim=True))
    x = state["x"].double() * spread(state["sx"].double(), (1, 128), *state["x"].shape)
    y = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
    for n in range(case["experts"]):
        rows = (at == n).any(1).nonzero()[:, 0]
        if not rows.numel():
            continue
        gate, up, down = (state[w][n].double() * spread(state["s_" + w][n].double(), (128, 128), *state[w].shape[1:]) for w in ("gate", "up", "down"))
        a = x[rows] @ gate.T
        y[rows] += p[rows, n][:, None] * ((a / (1.0 + torch.exp(-a)) * (x[rows] @ up.T)) @ down.T)
    return y


def unrounded(x, group, fmt):
    v = in_groups(x, group)
    s = (v.abs().amax(dim=(1, 3)) / F8_MAX[fmt]).clamp_min(TINY)
    q = v / s[:, None, :, None]
    return q.reshape(q.shape[0] * q.shape[1], -1)[: x.shape[0], : x.shape[1]], s


# ------------------------------------------------------------------ what a pass cannot do without

def groups_in(rows, cols, group):
    return -(-rows // group[0]) * -(-cols // group[1])


def work(case):
    op = case["op"]
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        ta, tb = case["ops"]
        scales = groups_in(*((K, M) if ta == "T" else (M, K)), GROUPS[case["group_a"]]) + groups_in(*((N, K) if tb == "T" else (K, N)), GROUPS[case["group_b"]])
        return {"bytes": M * K + K * N + 4 * scales + M * N * TYPE_BYTES[case["out"]] * (2 if case["beta"] else 1), "flops": 2.0 * M * N * K}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (TYPE_BYTES[case["type"]] + 1) + 4 * groups_in(case["rows"], case["cols"], GROUPS[case["group"]]), "flops": 3.0 * n}
    if op in ("norm", "norm_grad"):
        n, b = case["rows"] * case["cols"], TYPE_BYTES[case["type"]]
        if op == "norm":  # x, r, their sum and the codes
            return {"bytes": n * (b * (3 if case["residual"] else 1) + 1) + 4 * groups_in(case["rows"], case["cols"], (1, 128)) + 4 * case["rows"] + b * case["cols"], "flops": 8.0 * n}
        return {"bytes": n * b * (4 if case["residual"] else 3) + 4 * case["rows"] + (b + 4) * case["cols"], "flops": 10.0 * n}
    T, E, k, H, I = case["tokens"], case["experts"], case["top_k"], case["hidden"], case["inner"]
    hit = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token chose, on average
    return {"bytes": hit * 3 * H * I * (1 + 4 / 128 ** 2) + T * (H + 4 * E + 2 * H), "flops": 6.0 * T * k * H * I}
