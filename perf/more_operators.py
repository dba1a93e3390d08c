"""The gated feed-forward block of a training step as it is measured: cases, inputs, plain forms and the library's own calls.

Three operators, all over rows sorted by expert and split by a groupList (one group: a dense block, or a layer's shared expert):

- ``gated``: both projections, the activation and the product of the two in one call, ``h = act(x Wg) * (x Wu)``, with what the
  backward pass needs of the projections kept in 16 bits, in 8 (FP8 E4M3 codes, one E8M0 scale per 32 values) or not at all;
- ``back``: the gradient from behind the block's last projection, ``dh = dy Wd^T``, through the gate to both projections, and
  ``h`` again (for that projection's weight gradient), both from what was kept;
- ``wgrad``: the gradient of the weights where the rows that the forward pass multiplied were kept in 8 bits.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token through its eight experts, answering: nothing is kept
        dict(name="gated_token", op="gated", rows=8, experts=32, k=7168, f=2048, type="bf16", act="geglu", keep="none", turned=True, spread=0.0, list=1),
        # a training step's gate and up projections, kept in 8 bits for the backward pass
        dict(name="gated_step", op="gated", rows=32768, experts=32, k=7168, f=2048, type="bf16", act="swiglu", keep="fp8", turned=False, spread=0.0, list=0),
        # the shared expert, a dense block, kept in 16 bits
        dict(name="gated_shared", op="gated", rows=4096, experts=1, k=7168, f=2048, type="bf16", act="swiglu", keep="full", turned=True, spread=0.0, list=1),
        # small experts of odd sizes in half precision, some without rows
        dict(name="gated_ragged", op="gated", rows=6007, experts=48, k=1032, f=800, type="fp16", act="geglu", keep="fp8", turned=False, spread=1.2, list=1),
        # a short sequence, fine-tuned on a few experts
        dict(name="back_short", op="back", rows=64, experts=8, k=2048, f=1024, type="bf16", act="swiglu", keep="fp8", turned=False, spread=0.0, list=1),
        # the training step's way back, from what was kept in 8 bits
        dict(name="back_step", op="back", rows=32768, experts=32, k=7168, f=2048, type="bf16", act="swiglu", keep="fp8", turned=False, spread=0.0, list=0),
        # the shared expert's, from 16 bits
        dict(name="back_shared", op="back", rows=4096, experts=1, k=7168, f=2048, type="bf16", act="swiglu", keep="full", turned=True, spread=0.0, list=1),
        # the small experts'
        dict(name="back_ragged", op="back", rows=6007, experts=48, k=1032, f=800, type="fp16", act="geglu", keep="fp8", turned=True, spread=1.2, list=1),
        # the weights' gradient of the short sequence
        dict(name="wgrad_short", op="wgrad", rows=64, experts=8, k=2048, n=2048, type="bf16", out="bf16", turned=False, spread=0.0, list=1),
        # the training step's, in fp32 for the optimiser
        dict(name="wgrad_step", op="wgrad", rows=32768, experts=32, k=7168, n=4096, type="bf16", out="fp32", turned=False, spread=0.0, list=0),
        # weights kept as (e,n,k): the rows in 8 bits are the second operand
        dict(name="wgrad_turned", op="wgrad", rows=16384, experts=8, k=2048, n=4096, type="bf16", out="bf16", turned=True, spread=0.5, list=0),
        # the small experts'
        dict(name="wgrad_ragged", op="wgrad", rows=6007, experts=48, k=1088, n=1600, type="fp16", out="fp16", turned=False, spread=1.2, list=1),
    ]


def _log(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread evenly over the logarithm."""
    return min(hi // step, max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))) * step


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("gated", "back", "wgrad")}
    while True:
        op = rng.choice(["gated", "back", "wgrad"])
        case = dict(op=op, rows=_log(rng, 1, 65536, 1), experts=_log(rng, 1, 128, 1), type=rng.choice(["bf16", "fp16"]),
                    turned=rng.random() < 0.5, spread=round(rng.uniform(0, 1.5), 2), list=rng.randrange(2))
        if op == "wgrad":
            case.update(k=_log(rng, 128, 8192, 64), n=_log(rng, 128, 8192, 8), out=rng.choice(["fp32", case["type"]]))
        else:
            keep = rng.choice(["none", "full", "fp8"] if op == "gated" else ["full", "fp8"])
            case.update(k=_log(rng, 128, 8192, 8), f=_log(rng, 128, 4096, 32 if keep == "fp8" else 8), keep=keep, act=rng.choice(["swiglu", "geglu"]))
        if _cost(case) <= most[op] and case["experts"] * case["k"] * _columns(case) <= 1e9:
            return case


def _columns(case):
    """Columns of the weights beside the reduction or the rows' width k."""
    return {"gated": 2 * case.get("f", 0), "back": case.get("f", 0), "wgrad": case.get("n", 0)}[case["op"]]


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 5e12, w["flops"] / 1e15)


def _counts(case):
    """Rows of each expert, in an order of their own: `spread` is the exponent of their popularity's fall."""
    rng = random.Random("%d/%d/%s" % (case["rows"], case["experts"], case["spread"]))
    share = [(i + 1) ** -case["spread"] * rng.uniform(0.8, 1.2) for i in range(case["experts"])]
    exact_rows = [case["rows"] * s / sum(share) for s in share]
    counts = [int(r) for r in exact_rows]
    left = sorted(range(len(counts)), key=lambda i: counts[i] - exact_rows[i])[: case["rows"] - sum(counts)]
    for i in left:
        counts[i] += 1
    return counts


def work(case):
    rows, k, n = case["rows"], case["k"], _columns(case)
    busy = sum(c > 0 for c in _counts(case))
    flops = 2.0 * rows * k * n
    if case["op"] == "wgrad":
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": rows * (k * (1 + 1 / 32) + 2.0 * n) + case["experts"] * k * n * out, "flops": flops}
    f = case["f"]
    kept = rows * 2 * f * {"none": 0, "full": 2, "fp8": 1 + 1 / 32}[case["keep"]]
    if case["op"] == "gated":  # rows and weights in, h and what is kept out
        return {"bytes": 2.0 * (rows * k + busy * k * n + rows * f) + kept, "flops": flops}
    # dy, weights and what was kept in, the gradients of both projections and h out
    return {"bytes": 2.0 * (rows * k + busy * k * n + 3 * rows * f) + kept, "flops": flops}


# ---------------------------------------------------------------- inputs


def _normal(gen, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _hidden(gen, rows, k):
    """Hidden states: normal, with channels of unlike size and a few large ones."""
    channel = torch.exp(0.5 * torch.randn(k, generator=gen, device="cuda"))
    channel[torch.randint(0, k, (max(1, k // 256),), generator=gen, device="cuda")] *= 12.0
    return _normal(gen, rows, k).mul_(channel)


def _weights(gen, e, *shape, dtype, scale):
    w = torch.empty((e, *shape), dtype=dtype, device="cuda")
    for g in range(e):
        w[g] = _normal(gen, *shape, scale=scale)
    return w


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    counts = _counts(case)
    random.Random(seed).shuffle(counts)
    ends = [sum(counts[: g + 1]) for g in range(len(counts))]
    s = dict(case, counts=counts, groups=torch.tensor(ends if case["list"] == 0 else counts, dtype=torch.int64, device="cuda"))
    rows, e, k, n, dtype = case["rows"], case["experts"], case["k"], _columns(case), _TYPES[case["type"]]
    if case["op"] == "wgrad":
        s["x"], s["x_scale"] = _pack(*_encode(_hidden(gen, rows, k)))
        s["dy"] = _normal(gen, rows, n, dtype=dtype, scale=0.02)
        return s
    if case["op"] == "gated":
        s["x"] = (0.7 * _hidden(gen, rows, k)).to(dtype)
        s["w"] = _weights(gen, e, *((n, k) if case["turned"] else (k, n)), dtype=dtype, scale=k ** -0.5)
        return s
    s["dy"] = _normal(gen, rows, k, dtype=dtype, scale=0.02)
    s["w"] = _weights(gen, e, *((k, n) if case["turned"] else (n, k)), dtype=dtype, scale=n ** -0.5)
    kept = _normal(gen, rows, 2 * n, scale=1.5)
    s["kept"], s["kept_scale"] = _pack(*_encode(kept)) if case["keep"] == "fp8" else (kept.to(dtype), None)
    return s


# ---------------------------------------------------------------- plain forms


def _power(exponent):
    """2 to whole exponents in [-127, 127], in fp32 and exact."""
    return torch.where(exponent == -127, 1 << 22, (exponent + 127) << 23).to(torch.int32).view(torch.float32)


def _encode(x):
    """Blocks of 32 values along the last axis: each value over its block's power of two on the E4M3 grid, and the exponents."""
    x = x.unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    exponent = torch.where(top == 0, -127, (torch.frexp(top)[1].to(torch.int32) - 9).clamp(-127, 127))
    v = (x * _power(-exponent).unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    return v.flatten(-2), exponent


def _pack(v, exponent):
    """The stored form: E4M3 codes and E8M0 scales (..., k/64, 2)."""
    return v.to(torch.float8_e4m3fn), (exponent + 127).to(torch.uint8).unflatten(-1, (-1, 2)).contiguous().view(torch.float8_e8m0fnu)


def _values(code, scale):
    """The fp32 values that codes and scales stand for, or 16-bit ones widened."""
    if scale is None:
        return code.float()
    s = _power(scale.view(torch.uint8).int() - 127).flatten(-2)
    return (code.float().unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def _sigma(gate, act):
    """The factor that the activation puts on its gate, and the derivative of that factor's argument: silu is g / (1 + e^-g), and
    gelu in its tanh form g / (1 + e^-z) with z = sqrt(8 / pi) (g + 0.044715 g^3)."""
    if act == "swiglu":
        return 1 / (1 + torch.exp(-gate)), 1.0
    c = math.sqrt(8 / math.pi)
    return 1 / (1 + torch.exp(-c * (gate + 0.044715 * gate * gate * gate))), c * (1 + 3 * 0.044715 * gate * gate)


def _grouped(s, x, w, turned):
    """Each group's rows times its expert's weights, in fp32."""
    return torch.cat([p.float() @ (w[g].T if turned else w[g]).float() for g, p in enumerate(x.split(s["counts"])) if len(p)])


def _plain_gated(s):
    both = _grouped(s, s["x"], s["w"], s["turned"])
    gate, up = both.chunk(2, -1)
    out = {"h": (gate * _sigma(gate, s["act"])[0] * up).to(s["x"].dtype)}
    if s["keep"] == "full":
        out["kept"] = both.to(s["x"].dtype)
    elif s["keep"] == "fp8":
        v, exponent = _encode(both)
        out["kept"] = (v.unflatten(-1, (-1, 32)) * _power(exponent).unsqueeze(-1)).flatten(-2).to(torch.bfloat16)
    return out


def _plain_back(s):
    dh = _grouped(s, s["dy"], s["w"], not s["turned"])
    gate, up = _values(s["kept"], s["kept_scale"]).chunk(2, -1)
    sig, slope = _sigma(gate, s["act"])
    d_gate = dh * up * (sig + gate * sig * (1 - sig) * slope)
    return {"d": torch.cat((d_gate, dh * gate * sig), -1).to(s["dy"].dtype), "h": (gate * sig * up).to(s["dy"].dtype)}


def _plain_wgrad(s):
    x, dy = _values(s["x"], s["x_scale"]), s["dy"].float()
    a, b = (dy, x) if s["turned"] else (x, dy)
    return {"dw": torch.stack([p.T @ q for p, q in zip(a.split(s["counts"]), b.split(s["counts"]))]).to(_TYPES[s["out"]])}


# ---------------------------------------------------------------- the library's calls


def _own_gated(s):
    from quantized_moe_grouped_amd import binding as B
    h, kept, scale = B.gated_matmul(s["x"], s["w"], s["groups"], activation=s["act"], keep=None if s["keep"] == "none" else s["keep"],
                                    transpose_w=s["turned"], group_list_type=s["list"])
    if s["keep"] == "none":
        return {"h": h}
    return {"h": h, "kept": kept if scale is None else B.mx_dequantize(kept, scale, dtype=torch.bfloat16)}


def _own_back(s):
    from quantized_moe_grouped_amd import binding as B
    d, h = B.gated_matmul_backward(s["dy"], s["w"], s["groups"], s["kept"], kept_scale=s["kept_scale"], activation=s["act"],
                                   transpose_w=not s["turned"], group_list_type=s["list"])
    return {"d": d, "h": h}


def _own_wgrad(s):
    from quantized_moe_grouped_amd import binding as B
    if s["turned"]:
        return {"dw": B.grouped_matmul_wgrad(s["dy"], s["x"], s["groups"], dy_scale=s["x_scale"], out_dtype=_TYPES[s["out"]], group_list_type=s["list"])}
    return {"dw": B.grouped_matmul_wgrad(s["x"], s["dy"], s["groups"], x_scale=s["x_scale"], out_dtype=_TYPES[s["out"]], group_list_type=s["list"])}


def run(state):
    if own:
        return {"gated": _own_gated, "back": _own_back, "wgrad": _own_wgrad}[state["op"]](state)
    return {"gated": _plain_gated, "back": _plain_back, "wgrad": _plain_wgrad}[state["op"]](state)


# ---------------------------------------------------------------- the definition, in 64 bits


def _exact_power(exponent):
    """2 to whole exponents, put together from the fields of a 64-bit value (a library's pow may be off by a rounding)."""
    return ((exponent.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(code, scale):
    """E4M3 by its fields: (-1)^sign 2^(exponent - 7) (1 + mantissa / 8), subnormals without the 1; times the block's scale."""
    byte = code.view(torch.uint8).to(torch.int64)
    exponent, mantissa = (byte & 127) >> 3, (byte & 7).double() / 8
    v = torch.where(exponent == 0, mantissa * 2.0 ** -6, (1 + mantissa) * _exact_power(exponent - 7))
    v = torch.where(byte >= 128, -v, v)
    return v * _exact_power(scale.view(torch.uint8).to(torch.int64) - 127).reshape(v.shape[0], -1).repeat_interleave(32, -1)


def _exact_rounded(x):
    """x on the grid of its block of 32: E4M3 steps over the power of two that brings the block's largest value under 512."""
    shape = x.shape
    x = x.reshape(shape[0], -1, 32)
    mantissa, exponent = torch.frexp(x.abs().max(-1, keepdim=True).values)
    size = _exact_power(torch.where(mantissa == 0, torch.full_like(exponent, -127), exponent - 9).clamp(-127, 127))
    v = x / size
    step = _exact_power((torch.frexp(v.abs())[1] - 1).clamp(min=-6) - 3)
    return ((torch.round(v / step) * step).clamp(-448, 448) * size).reshape(shape)


def _exact_gate(g, act):
    """Activation and derivative. silu(g) = g / (1 + e^-g); gelu(g) = g/2 (1 + tanh t), t = sqrt(2/pi) (g + 0.044715 g^3)."""
    if act == "swiglu":
        e = torch.exp(-g)
        return g / (1 + e), (1 + e + g * e) / (1 + e) ** 2
    c = (2 / math.pi) ** 0.5
    th = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)


def exact(case, seed):
    s = prepare(case, seed)
    starts = [0]
    for c in s["counts"]:
        starts.append(starts[-1] + c)
    k, n, rows = case["k"], _columns(case), case["rows"]
    if case["op"] == "wgrad":
        x = _exact_values(s["x"], s["x_scale"])
        dw = torch.zeros((case["experts"], n, k) if case["turned"] else (case["experts"], k, n), dtype=torch.float64, device="cuda")
        for g, c in enumerate(s["counts"]):
            if c:
                part = slice(starts[g], starts[g + 1])
                a, b = x[part], s["dy"][part].double()
                dw[g] = torch.mm(b.T.contiguous(), a) if case["turned"] else torch.mm(a.T.contiguous(), b)
        return {"dw": dw}
    y = torch.empty((rows, n), dtype=torch.float64, device="cuda")
    x = s["x"] if case["op"] == "gated" else s["dy"]
    along = case["turned"] == (case["op"] == "gated")  # weights stored with the reduction last
    for g, c in enumerate(s["counts"]):
        if c:
            part, w = slice(starts[g], starts[g + 1]), s["w"][g].double()
            y[part] = torch.mm(x[part].double(), w.T if along else w)
    if case["op"] == "gated":
        out = {"h": _exact_gate(y[:, : n // 2], case["act"])[0] * y[:, n // 2 :]}
        if case["keep"] != "none":
            out["kept"] = y if case["keep"] == "full" else _exact_rounded(y)
        return out
    both = s["kept"].double() if s["kept_scale"] is None else _exact_values(s["kept"], s["kept_scale"])
    a, slope = _exact_gate(both[:, :n], case["act"])
    up = both[:, n:]
    return {"d": torch.cat((y * up * slope, y * a), -1), "h": a * up}
