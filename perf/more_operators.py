"""The operators on BF16 layers of libsgemm as cases that can be timed and compared.

Each case runs one operator on inputs made from a seed: with ``own`` false in
plain torch operations (32-bit arithmetic whatever the inputs' type, one
rounding at the end), with ``own`` true through the calls a user of
``sgemm_row_major_gb300`` makes.  ``exact`` gives the same outputs from the
operator's definition in 64 bits.

Operators:

* ``linear``       y = act(x W^T + bias) + residual, and what the backward pass wants of x W^T + bias: BF16 or 8-bit codes with scales
* ``linear_grad``  its backward pass from either
* ``gated``        h = act(x G^T) * (x U^T), and what the backward pass wants of both products
* ``gated_grad``   its backward pass
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TYPE_BYTES = {"f32": 4, "bf16": 2}
ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")
SAVE = ("none", "bf16", "fp8")
GROUP, TOP = 128, 448.0  # 8-bit values: E4M3 codes with a scale per 128 elements of a row
TINY = 2.0 ** -126       # the smallest scale


def listed():
    return [
        # one token through a square layer, added to the stream that bypasses it: the call of every decoding step, all latency and weight bytes
        linear("linear 1x4096x4096", 1, 4096, 4096, residual=True),
        # a batch of 64 decoding sequences through a wide layer (a fully connected shape of the library's own benchmark)
        linear("linear 64x16384x4096", 64, 16384, 4096, bias=True, act="gelu"),
        # no size a multiple of anything and rows of odd lengths one behind the other: the ragged shape of the library's own benchmark
        linear("linear 4097x2053x3001", 4097, 2053, 3001, bias=True, act="gelu", residual=True, packed=True),
        # a training batch through a widening layer, which keeps what its backward pass wants in 8 bits
        linear("linear 8192x4096x16384", 8192, 4096, 16384, bias=True, act="gelu_tanh", save="fp8"),
        # the gradients of a small layer of uneven sizes
        linear_grad("linear gradient 1000x1300x700", 1000, 1300, 700, act="relu", save="bf16", dbias=True),
        # the gradients of a layer without an activation, the weights' in FP32
        linear_grad("linear gradient 8192x4096x4096", 8192, 4096, 4096, dw="f32"),
        # the gradients of the widening layer from what it kept in 8 bits
        linear_grad("linear gradient 4096x4096x16384", 4096, 4096, 16384, act="gelu_tanh", save="fp8", dbias=True),
        # one token through the first half of a gated feed-forward block
        gated("gated 1x4096x8192", 1, 4096, 8192),
        # 64 decoding sequences through the same of a small model
        gated("gated 64x2048x1024", 64, 2048, 1024),
        # a training batch, both products kept in 8 bits
        gated("gated 8192x4096x8192", 8192, 4096, 8192, save="fp8"),
        # the gradients at uneven sizes, both products kept as they were
        gated("gated gradient 1000x1300x700", 1000, 1300, 700, act="gelu", save="bf16", op="gated_grad"),
        # the gradients of the training batch from 8 bits, and h again for the weight gradient of the layer behind: the largest call
        dict(gated("gated gradient 8192x4096x8192", 8192, 4096, 8192, save="fp8", op="gated_grad"), again=True),
    ]


def linear(name, tokens, inputs, outputs, bias=False, act="none", residual=False, save="none", out="bf16", packed=False):
    return {"name": name, "op": "linear", "tokens": tokens, "inputs": inputs, "outputs": outputs, "bias": bias, "act": act, "residual": residual,
            "save": save, "out": out, "packed": packed}


def linear_grad(name, tokens, inputs, outputs, act="none", save="none", dbias=False, dw="bf16", packed=False):
    return {"name": name, "op": "linear_grad", "tokens": tokens, "inputs": inputs, "outputs": outputs, "act": act, "save": save, "dbias": dbias,
            "dw": dw, "packed": packed}


def gated(name, tokens, inputs, outputs, act="silu", save="none", packed=False, op="gated"):
    return {"name": name, "op": op, "tokens": tokens, "inputs": inputs, "outputs": outputs, "act": act, "save": save, "again": False, "packed": packed}


# ------------------------------------------------------------------ drawn cases

PRODUCTS = {"linear": 1, "linear_grad": 2, "gated": 2, "gated_grad": 6}  # of tokens x inputs x outputs


def between(rng, low, high):
    """A size spread over the logarithm of [low, high]; one in three is a power of two."""
    if rng.random() < 0.33:
        return rng.choice([2 ** k for k in range(15) if low <= 2 ** k <= high])
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "gated", "gated_grad"])
    while True:
        T, I, O = between(rng, 1, 16384), between(rng, 64, 16384), between(rng, 64, 16384)
        if PRODUCTS[op] * T * I * O <= 6 * 8192 * 4096 * 8192:
            break
    packed = rng.random() < 0.25
    if op == "linear":
        c = linear("", T, I, O, rng.random() < 0.5, rng.choice(ACTIVATIONS), rng.random() < 0.5, rng.choice(SAVE), rng.choice(["bf16", "bf16", "f32"]), packed)
    elif op == "linear_grad":
        act = rng.choice(ACTIVATIONS)
        c = linear_grad("", T, I, O, act, rng.choice(SAVE[1:]) if act != "none" else "none", rng.random() < 0.5, "bf16" if act != "none" else rng.choice(["bf16", "f32"]), packed)
    else:
        c = gated("", T, I, O, rng.choice(ACTIVATIONS), rng.choice(SAVE if op == "gated" else SAVE[1:]), packed, op)
        c["again"] = op == "gated_grad" and rng.random() < 0.5
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def normal(g, rows, cols, std=1.0):
    return torch.randn(rows, cols, generator=g, device="cuda") * std


def activations(g, rows, cols):
    """Values as they leave a layer: near normal, with a few columns much larger than the rest."""
    loud = torch.rand(cols, generator=g, device="cuda") < 0.01
    return normal(g, rows, cols) * torch.where(loud, 12.0, 1.0)


def stored(x, packed, dtype=torch.bfloat16):
    """x as a matrix in memory: rows one behind the other, or starting at multiples of 16 elements."""
    rows, cols = x.shape
    ld = cols if packed else (cols + 15) // 16 * 16
    m = torch.zeros(rows, ld, dtype=dtype, device="cuda")[:, :cols]
    m.copy_(x)
    return m


def in_groups(x):
    """x, its rows padded by zeros to whole groups, seen as [rows, groups, 128]."""
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % GROUP))
    return x.view(x.shape[0], -1, GROUP)


def codes_of(x):
    """8-bit codes of x and the scales of its groups."""
    v = in_groups(x)
    s = (v.abs().amax(2) / TOP).clamp_min(TINY)
    q = (v * (1.0 / s)[:, :, None]).clamp(-TOP, TOP)
    return q.view(x.shape[0], -1)[:, : x.shape[1]].to(torch.float8_e4m3fn), s


def kept(x, how, packed):
    """What a forward pass kept of x for its backward pass: a matrix, or codes and scales."""
    if how == "bf16":
        return stored(x, packed)
    q, s = codes_of(x)
    rows, cols = x.shape
    ld = cols if packed else (cols + 15) // 16 * 16
    m = torch.zeros(rows, ld, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :cols]
    m.view(torch.uint8).copy_(q.contiguous().view(torch.uint8))
    return m, s


def value(k, dtype=torch.float32):
    """The numbers that a kept matrix stands for."""
    if torch.is_tensor(k):
        return k.to(dtype)
    q, s = k
    return q.to(dtype) * s.to(dtype).repeat_interleave(GROUP, 1)[:, : q.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    T, I, O, op, packed = case["tokens"], case["inputs"], case["outputs"], case["op"], case["packed"]
    state = {"case": case, "x": stored(activations(g, T, I), packed)}
    for key in ("w",) if op in ("linear", "linear_grad") else ("gate", "up"):
        state[key] = stored(normal(g, O, I, I ** -0.5), packed)
    if op == "linear":
        state["bias"] = normal(g, 1, O, 0.5)[0].to(torch.bfloat16) if case["bias"] else None
        state["residual"] = stored(activations(g, T, O), packed) if case["residual"] else None
    elif op == "linear_grad":
        state["dy"] = stored(normal(g, T, O, 1e-2), packed)
        state["pre"] = kept(normal(g, T, O), case["save"], packed) if case["save"] != "none" else None
    elif op == "gated_grad":
        state["dh"] = stored(normal(g, T, O, 1e-2), packed)
        state["gate_pre"], state["up_pre"] = (kept(normal(g, T, O), case["save"], packed) for _ in range(2))
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    return (own_run if own else plain_run)(state)


def own_run(state):
    import sgemm_row_major_gb300 as sg

    def given(k):
        return k if k is None or torch.is_tensor(k) else sg.Fp8Matrix(*k)

    def parts(name, k):
        if k is None:
            return {}
        return {name: k} if torch.is_tensor(k) else {name + "_codes": k.data, name + "_scale": k.scale}

    case, op = state["case"], state["case"]["op"]
    act = None if case["act"] == "none" else case["act"]
    save = None if case["save"] == "none" else case["save"]
    if op == "linear":
        got = sg.linear_bf16(state["x"], state["w"], state["bias"], act, state["residual"], save=save, out_dtype=TYPES[case["out"]])
        return {"y": got.y} | parts("pre", got.pre)
    if op == "linear_grad":
        got = sg.linear_bf16_backward(state["dy"], state["x"], state["w"], given(state["pre"]), act, dbias=case["dbias"], dweight_dtype=TYPES[case["dw"]])
        return {"dx": got.dx, "dw": got.dweight} | parts("dbias", got.dbias)
    if op == "gated":
        got = sg.gated_bf16(state["x"], state["gate"], state["up"], act, save=save)
        return {"h": got.h} | parts("gate", got.gate) | parts("up", got.up)
    got = sg.gated_bf16_backward(state["dh"], state["x"], state["gate"], state["up"], given(state["gate_pre"]), given(state["up_pre"]), act, h=case["again"])
    return {"dx": got.dx, "dgate": got.dgate, "dup": got.dup} | parts("h", got.h)


def plain_act(a, act):
    """The activation and its derivative."""
    if act == "none":
        return a, torch.ones_like(a)
    if act == "relu":
        on = (a > 0).to(a.dtype)
        return a * on, on
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-a))
        return a * s, s * (1.0 + a * (1.0 - s))
    if act == "gelu":
        c = 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5)))
        return a * c, c + a * torch.exp(-0.5 * a * a) * (1.0 / math.sqrt(2.0 * math.pi))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (a + 0.044715 * a * a * a))
    return 0.5 * a * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * a * a)


def plain_kept(name, v, how):
    if how == "none":
        return {}
    if how == "bf16":
        return {name: v.to(torch.bfloat16)}
    q, s = codes_of(v)
    return {name + "_codes": q, name + "_scale": s}


def plain_run(state):
    case, op, x = state["case"], state["case"]["op"], state["x"].float()
    if op == "linear":
        pre = x @ state["w"].float().T
        if state["bias"] is not None:
            pre = pre + state["bias"].float()
        y = plain_act(pre, case["act"])[0]
        if state["residual"] is not None:
            y = y + state["residual"].float()
        return {"y": y.to(TYPES[case["out"]])} | plain_kept("pre", pre, case["save"])
    if op == "linear_grad":
        d = state["dy"].float()
        if state["pre"] is not None:
            d = d * plain_act(value(state["pre"]), case["act"])[1]
        got = {"dx": (d @ state["w"].float()).to(torch.bfloat16), "dw": (d.T @ x).to(TYPES[case["dw"]])}
        return got | ({"dbias": d.sum(0)} if case["dbias"] else {})
    if op == "gated":
        a, b = x @ state["gate"].float().T, x @ state["up"].float().T
        return {"h": (plain_act(a, case["act"])[0] * b).to(torch.bfloat16)} | plain_kept("gate", a, case["save"]) | plain_kept("up", b, case["save"])
    dh, a, b = state["dh"].float(), value(state["gate_pre"]), value(state["up_pre"])
    f, df = plain_act(a, case["act"])
    da, db = dh * b * df, dh * f
    got = {"dx": da @ state["gate"].float() + db @ state["up"].float(), "dgate": da.T @ x, "dup": db.T @ x}
    if case["again"]:
        got["h"] = f * b
    return {k: v.to(torch.bfloat16) for k, v in got.items()}


# ------------------------------------------------------------------ 64 bits

def exact_act(a, act):
    f = torch.nn.functional
    return {"none": lambda v: v, "relu": f.relu, "silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[act](a)


def exact_kept(name, v, how):
    """Codes are given before their rounding to 8 bits (a value over its scale): one next to a tie goes either way, but its
    distance from the unrounded one is the type's."""
    if how == "none":
        return {}
    if how == "bf16":
        return {name: v}
    s = (in_groups(v).abs().amax(2) / TOP).clamp_min(TINY)
    return {name + "_codes": v / s.repeat_interleave(GROUP, 1)[:, : v.shape[1]], name + "_scale": s}


def exact(case, seed):
    """run()'s outputs from the definitions in 64 bits, the gradients by differentiating the forward pass."""
    state = prepare(case, seed)
    op, act = case["op"], case["act"]
    x = state["x"].double()
    if op == "linear":
        pre = torch.einsum("ti,oi->to", x, state["w"].double()) + (0.0 if state["bias"] is None else state["bias"].double()[None])
        y = exact_act(pre, act) + (0.0 if state["residual"] is None else state["residual"].double())
        return {"y": y} | exact_kept("pre", pre, case["save"])
    if op == "gated":
        a, b = (torch.einsum("ti,oi->to", x, state[k].double()) for k in ("gate", "up"))
        return {"h": exact_act(a, act) * b} | exact_kept("gate", a, case["save"]) | exact_kept("up", b, case["save"])
    if op == "linear_grad":
        d = state["dy"].double()
        if state["pre"] is not None:
            pre = value(state["pre"], torch.float64).requires_grad_()
            d, = torch.autograd.grad(exact_act(pre, act), pre, d)
        got = {"dx": torch.einsum("to,oi->ti", d, state["w"].double()), "dw": torch.einsum("to,ti->oi", d, x)}
        return got | ({"dbias": d.sum(0)} if case["dbias"] else {})
    a, b = (value(state[k], torch.float64).requires_grad_() for k in ("gate_pre", "up_pre"))
    h = exact_act(a, act) * b
    da, db = torch.autograd.grad(h, (a, b), state["dh"].double())
    got = {"dx": torch.einsum("to,oi->ti", da, state["gate"].double()) + torch.einsum("to,oi->ti", db, state["up"].double()),
           "dgate": torch.einsum("to,ti->oi", da, x), "dup": torch.einsum("to,ti->oi", db, x)}
    return got | ({"h": h.detach()} if case["again"] else {})


# ------------------------------------------------------------------ what a pass cannot do without

def kept_bytes(T, O, how):
    return {"none": 0, "bf16": 2 * T * O, "fp8": T * O + 4 * T * -(-O // GROUP)}[how]


def work(case):
    T, I, O, op = case["tokens"], case["inputs"], case["outputs"], case["op"]
    k = kept_bytes(T, O, case["save"])
    if op == "linear":
        n = 2 * (T * I + O * I) + T * O * TYPE_BYTES[case["out"]] + k + (2 * T * O if case["residual"] else 0) + (2 * O if case["bias"] else 0)
    elif op == "linear_grad":
        n = 2 * (T * O + T * I + O * I) + k + 2 * T * I + O * I * TYPE_BYTES[case["dw"]] + (4 * O if case["dbias"] else 0)
    elif op == "gated":
        n = 2 * (T * I + 2 * O * I + T * O) + 2 * k
    else:
        n = 2 * (T * O + T * I + 2 * O * I) + 2 * k + 2 * (T * I + 2 * O * I) + (2 * T * O if case["again"] else 0)
    return {"bytes": n, "flops": 2.0 * PRODUCTS[op] * T * I * O}
