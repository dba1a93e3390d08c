"""The expert layer's operators as they are measured: cases, inputs, plain forms and the library's own calls.

Four operators, all over rows sorted by expert and split by a groupList:

- ``quant``: microscaled quantisation (FP4 E2M1 or FP8 E4M3 codes, one E8M0 scale per 32 values) and back to values;
- ``mx``: products grouped by expert of microscaled operands, FP4 or FP8 rows with FP4 weights, plain or with SwiGLU;
- ``dense``: the same products of 16-bit operands, with the weights as stored or transposed (the gradient of the rows);
- ``wgrad``: the gradient of the weights, one product of rows with rows for each expert.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step's hidden states, eight tokens: latency
        dict(name="quant_tokens", op="quant", experts=1, rows=8, k=7168, type="bf16", format="fp4", turned=False),
        # a prefill batch's hidden states, quantised before the expert products
        dict(name="quant_prefill", op="quant", experts=1, rows=16384, k=7168, type="bf16", format="fp8", turned=False),
        # a checkpoint's weights (e,k,n), brought to the FP4 products' (e,n,k) layout when they are loaded
        dict(name="quant_weights", op="quant", experts=32, rows=7168, k=2048, type="bf16", format="fp4", turned=True),
        # one token through its eight experts' gate and up projections
        dict(name="mx_token", op="mx", rows=8, experts=32, k=7168, n=4096, x="fp4", act="swiglu", spread=0.0, list=1),
        # a decode batch over very many experts, a few taking most rows and others none
        dict(name="mx_skewed", op="mx", rows=2048, experts=256, k=2048, n=7168, x="fp8", act="none", spread=1.2, list=0),
        # prefill: the gate and up projections of 16384 tokens, eight experts each
        dict(name="mx_prefill", op="mx", rows=131072, experts=32, k=7168, n=4096, x="fp4", act="swiglu", spread=0.0, list=1),
        # a middling batch with FP8 rows, sizes that end inside every tile
        dict(name="mx_ragged", op="mx", rows=30001, experts=64, k=2112, n=7152, x="fp8", act="none", spread=0.4, list=0),
        # one token through unquantised experts
        dict(name="dense_token", op="dense", rows=8, experts=32, k=2048, n=7168, type="bf16", turned=True, spread=0.0, list=1),
        # the down projection of a training step, weights (e,k,n)
        dict(name="dense_step", op="dense", rows=32768, experts=32, k=2048, n=7168, type="bf16", turned=False, spread=0.0, list=0),
        # its gradient towards the rows, the same weights transposed; ragged sizes, half precision
        dict(name="dense_back", op="dense", rows=20011, experts=64, k=7160, n=2040, type="fp16", turned=True, spread=0.6, list=1),
        # its gradient towards the weights, summed in fp32 for the optimiser
        dict(name="wgrad_step", op="wgrad", rows=32768, experts=32, k=2048, n=7168, type="bf16", out="fp32", spread=0.0, list=0),
        # small experts of odd sizes, a few long ones among them, some without rows
        dict(name="wgrad_ragged", op="wgrad", rows=6007, experts=48, k=1032, n=776, type="fp16", out="fp16", spread=1.2, list=1),
    ]


def _log(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread evenly over the logarithm."""
    return min(hi // step, max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))) * step


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("quant", "mx", "dense", "wgrad")}
    while True:
        op = rng.choice(["quant", "mx", "dense", "wgrad"])
        if op == "quant":
            turned = rng.random() < 0.4
            case = dict(op=op, experts=_log(rng, 1, 64, 1) if turned else 1,
                        rows=_log(rng, 8, 8192, 8) if turned else _log(rng, 1, 131072, 1), k=_log(rng, 64, 8192, 64),
                        type=rng.choice(["bf16", "fp16", "fp32"]), format=rng.choice(["fp4", "fp8"]), turned=turned)
        else:
            rows, experts = _log(rng, 1, 131072, 1), _log(rng, 1, 256, 1)
            case = dict(op=op, rows=rows, experts=experts, spread=round(rng.uniform(0, 1.5), 2), list=rng.randrange(2))
            if op == "mx":
                act = rng.choice(["none", "swiglu"])
                case.update(k=_log(rng, 256, 8192, 64), n=_log(rng, 256, 8192, 16), x=rng.choice(["fp4", "fp8"]), act=act)
            else:
                case.update(k=_log(rng, 256, 8192, 8), n=_log(rng, 256, 8192, 8), type=rng.choice(["bf16", "fp16"]))
                case.update(dict(turned=rng.random() < 0.5) if op == "dense" else dict(out=rng.choice(["fp32", case["type"]])))
        if _cost(case) <= most[op] and case.get("experts", 1) * case["k"] * case.get("n", 1) <= 4e9:
            return case


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
    if case["op"] == "quant":
        values = case["experts"] * case["rows"] * case["k"]
        code = 0.5 if case["format"] == "fp4" else 1.0
        size = 4 if case["type"] == "fp32" else 2
        # in, codes and scales out; codes and scales in, values out
        return {"bytes": values * (size + 2 * code + 2 / 32 + 2), "flops": 0}
    rows, k, n = case["rows"], case["k"], case["n"]
    busy = sum(c > 0 for c in _counts(case))
    flops = 2.0 * rows * k * n
    if case["op"] == "mx":
        row = k * ((0.5 if case["x"] == "fp4" else 1.0) + 1 / 32)
        return {"bytes": rows * row + busy * n * k * (0.5 + 1 / 32) + rows * n * (1 if case["act"] == "swiglu" else 2), "flops": flops}
    if case["op"] == "dense":
        return {"bytes": 2.0 * (rows * k + busy * k * n + rows * n), "flops": flops}
    return {"bytes": 2.0 * rows * (k + n) + case["experts"] * k * n * (4 if case["out"] == "fp32" else 2), "flops": flops}


# ---------------------------------------------------------------- inputs


def _normal(gen, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _hidden(gen, rows, k, dtype):
    """Hidden states: normal, with channels of unlike size and a few large ones."""
    channel = torch.exp(0.5 * torch.randn(k, generator=gen, device="cuda"))
    channel[torch.randint(0, k, (max(1, k // 256),), generator=gen, device="cuda")] *= 12.0
    return _normal(gen, rows, k).mul_(channel).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "quant":
        dtype = _TYPES[case["type"]]
        if case["turned"]:
            x = torch.empty((case["experts"], case["k"], case["rows"]), dtype=dtype, device="cuda")
            for g in range(case["experts"]):
                x[g] = _normal(gen, case["k"], case["rows"], scale=case["k"] ** -0.5)
        else:
            x = _hidden(gen, case["rows"], case["k"], dtype)
        return dict(case, x=x)
    counts = _counts(case)
    random.Random(seed).shuffle(counts)
    ends = [sum(counts[: g + 1]) for g in range(len(counts))]
    state = dict(case, counts=counts, groups=torch.tensor(ends if case["list"] == 0 else counts, dtype=torch.int64, device="cuda"))
    rows, e, k, n = case["rows"], case["experts"], case["k"], case["n"]
    if case["op"] == "mx":
        fmt = case["x"]
        state["x"], state["x_scale"] = _pack(*_encode(_hidden(gen, rows, k, torch.float32) * 0.7, fmt), fmt)
        w = torch.empty((e, n, k // 2), dtype=torch.uint8, device="cuda")
        s = torch.empty((e, n, k // 64, 2), dtype=torch.uint8, device="cuda")
        for g in range(e):
            code, scale = _pack(*_encode(_normal(gen, n, k, scale=k ** -0.5), "fp4"), "fp4")
            w[g], s[g] = code.view(torch.uint8), scale.view(torch.uint8)
        state["w"], state["w_scale"] = w.view(torch.float4_e2m1fn_x2), s.view(torch.float8_e8m0fnu)
        return state
    dtype = _TYPES[case["type"]]
    state["x"] = _normal(gen, rows, k, dtype=dtype)
    if case["op"] == "wgrad":
        state["dy"] = _normal(gen, rows, n, dtype=dtype, scale=0.02)
        return state
    w = torch.empty((e, n, k) if case["turned"] else (e, k, n), dtype=dtype, device="cuda")
    for g in range(e):
        w[g] = _normal(gen, *w.shape[1:], scale=k ** -0.5)
    state["w"] = w
    return state


# ---------------------------------------------------------------- plain forms

_FP4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _power(exponent):
    """2 to whole exponents in [-127, 127], in fp32 and exact."""
    return torch.where(exponent == -127, 1 << 22, (exponent + 127) << 23).to(torch.int32).view(torch.float32)


def _encode(x, fmt):
    """Blocks of 32 values along the last axis: the block's exponent, and each value over it on the format's grid."""
    x = x.float().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    exponent = torch.frexp(top)[1].to(torch.int32) - 1 - (2 if fmt == "fp4" else 8)
    exponent = torch.where(top == 0, -127, exponent.clamp(-127, 127))
    v = x * _power(-exponent).unsqueeze(-1)
    if fmt == "fp8":
        v = v.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    else:
        a = v.abs()  # nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code
        a = 0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75) + (a > 2.5) + (a >= 3.5) + 2.0 * (a > 5)
        v = torch.copysign(a, v)
    return v.flatten(-2), exponent


def _pack(v, exponent, fmt):
    """The stored form: codes (FP4 two per byte, the lower first) and E8M0 scales (..., k/64, 2)."""
    scale = (exponent + 127).to(torch.uint8).unflatten(-1, (-1, 2)).contiguous().view(torch.float8_e8m0fnu)
    if fmt == "fp8":
        return v.to(torch.float8_e4m3fn), scale
    a = v.abs()
    code = sum((a >= t).to(torch.uint8) for t in _FP4[1:]) + 8 * torch.signbit(v).to(torch.uint8)
    return (code[..., 0::2] + 16 * code[..., 1::2]).view(torch.float4_e2m1fn_x2), scale


def _values(code, scale):
    """The fp32 values that codes and scales stand for."""
    if code.dtype == torch.float8_e4m3fn:
        v = code.float()
    else:
        both = torch.tensor(_FP4 + [-f for f in _FP4], device=code.device)
        byte = code.view(torch.uint8).int()
        v = torch.stack((both[byte & 15], both[byte >> 4]), -1).flatten(-2)
    s = _power(scale.view(torch.uint8).int() - 127).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def _plain_quant(s):
    x = s["x"].transpose(1, 2).contiguous() if s["turned"] else s["x"]
    v, exponent = _encode(x, s["format"])
    scale = _power(exponent)
    return {"values": (v.unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2).to(torch.bfloat16),
            "scales": scale.unflatten(-1, (-1, 2))}


def _plain_mx(s):
    x = _values(s["x"], s["x_scale"]).split(s["counts"])
    # float4 tensors have no indexing of their own
    w, scale = s["w"].view(torch.uint8), s["w_scale"].view(torch.uint8)
    y = torch.cat([part @ _values(w[g].view(torch.float4_e2m1fn_x2), scale[g]).T for g, part in enumerate(x) if len(part)])
    if s["act"] == "swiglu":
        gate, up = y.chunk(2, -1)
        y = gate / (1 + torch.exp(-gate)) * up
    return {"y": y.to(torch.bfloat16)}


def _plain_dense(s):
    w = s["w"].transpose(1, 2) if s["turned"] else s["w"]
    y = torch.cat([part.float() @ w[g].float() for g, part in enumerate(s["x"].split(s["counts"])) if len(part)])
    return {"y": y.to(s["x"].dtype)}


def _plain_wgrad(s):
    parts = zip(s["x"].split(s["counts"]), s["dy"].split(s["counts"]))
    return {"dw": torch.stack([x.float().T @ dy.float() for x, dy in parts]).to(_TYPES[s["out"]])}


# ---------------------------------------------------------------- the library's calls


def _own_quant(s):
    from quantized_moe_grouped_amd import binding as B
    code, scale = B.mx_quantize(s["x"], format=s["format"], transpose=s["turned"])
    return {"values": B.mx_dequantize(code, scale, dtype=torch.bfloat16), "scales": scale.float()}


def _own_mx(s):
    from quantized_moe_grouped_amd import binding as B
    return {"y": B.grouped_matmul(s["x"], s["w"], s["groups"], x_scale=s["x_scale"], w_scale=s["w_scale"], transpose_w=True,
                                  activation=s["act"], out_dtype=torch.bfloat16, group_list_type=s["list"])}


def _own_dense(s):
    from quantized_moe_grouped_amd import binding as B
    return {"y": B.grouped_matmul(s["x"], s["w"], s["groups"], transpose_w=s["turned"], group_list_type=s["list"])}


def _own_wgrad(s):
    from quantized_moe_grouped_amd import binding as B
    return {"dw": B.grouped_matmul_wgrad(s["x"], s["dy"], s["groups"], out_dtype=_TYPES[s["out"]], group_list_type=s["list"])}


def run(state):
    if own:
        return {"quant": _own_quant, "mx": _own_mx, "dense": _own_dense, "wgrad": _own_wgrad}[state["op"]](state)
    return {"quant": _plain_quant, "mx": _plain_mx, "dense": _plain_dense, "wgrad": _plain_wgrad}[state["op"]](state)


# ---------------------------------------------------------------- the definition, in 64 bits


def _exact_values(code, scale, k):
    """Values from the formats' fields: (-1)^sign 2^(exponent - bias) (1 + mantissa / 2^bits), subnormals without the 1."""
    byte = code.view(torch.uint8).to(torch.int64)
    if code.dtype == torch.float8_e4m3fn:
        field, bits, bias = byte, 3, 7
    else:
        field, bits, bias = torch.empty((*byte.shape[:-1], k), dtype=torch.int64, device=byte.device), 1, 1
        field[..., 0::2], field[..., 1::2] = byte % 16, byte // 16
    sign, rest = field >> (7 if bits == 3 else 3), field & (127 if bits == 3 else 7)
    exponent, mantissa = rest >> bits, (rest & ((1 << bits) - 1)).double() / (1 << bits)
    v = torch.where(exponent == 0, mantissa * 2.0 ** (1 - bias), (1 + mantissa) * _exact_power(exponent - bias))
    block = _exact_power(scale.view(torch.uint8).to(torch.int64) - 127).reshape(*v.shape[:-1], k // 32)
    return torch.where(sign == 1, -v, v) * block.repeat_interleave(32, -1)


def _exact_power(exponent):
    """2 to whole exponents, put together from the fields of a 64-bit value (a library's pow may be off by a rounding)."""
    return ((exponent.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_quant(x, fmt):
    shape = x.shape
    x = x.double().reshape(-1, shape[-1] // 32, 32)
    top = x.abs().max(-1, keepdim=True).values
    mantissa, exponent = torch.frexp(top)  # top = mantissa * 2^exponent, mantissa in [0.5, 1)
    s = torch.where(mantissa == 0, torch.full_like(exponent, -127), exponent - (3 if fmt == "fp4" else 9)).clamp(-127, 127)
    size = _exact_power(s)
    v = x / size
    low, most = (0, 6.0) if fmt == "fp4" else (-6, 448.0)
    fine = 1 if fmt == "fp4" else 3
    step = _exact_power((torch.frexp(v.abs())[1] - 1).clamp(min=low) - fine)
    v = (torch.round(v / step) * step).clamp(-most, most)
    return (v * size).reshape(shape), size.reshape(*shape[:-1], -1, 2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        x = s["x"].movedim(1, 2).contiguous() if case["turned"] else s["x"].unsqueeze(0)
        parts = [_exact_quant(one, case["format"]) for one in x]
        values, scales = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
        return {"values": values, "scales": scales} if case["turned"] else {"values": values[0], "scales": scales[0]}
    starts = [0]
    for c in s["counts"]:
        starts.append(starts[-1] + c)
    k, n = case["k"], case["n"]
    if case["op"] == "wgrad":
        dw = torch.zeros((case["experts"], k, n), dtype=torch.float64, device="cuda")
        for g, c in enumerate(s["counts"]):
            if c:
                rows = slice(starts[g], starts[g + 1])
                dw[g] = torch.mm(s["x"][rows].double().T.contiguous(), s["dy"][rows].double())
        return {"dw": dw}
    y = torch.empty((case["rows"], n), dtype=torch.float64, device="cuda")
    for g, c in enumerate(s["counts"]):
        if not c:
            continue
        rows = slice(starts[g], starts[g + 1])
        if case["op"] == "dense":
            w = s["w"][g].double()
            y[rows] = torch.mm(s["x"][rows].double(), w.T if case["turned"] else w)
        else:
            x = _exact_values(s["x"].view(torch.uint8)[rows].view(s["x"].dtype), s["x_scale"].view(torch.uint8)[rows], k)
            w = _exact_values(s["w"].view(torch.uint8)[g].view(s["w"].dtype), s["w_scale"].view(torch.uint8)[g], k)
            y[rows] = torch.mm(x, w.T)
    if case.get("act") == "swiglu":
        return {"y": y[:, : n // 2] * torch.sigmoid(y[:, : n // 2]) * y[:, n // 2 :]}
    return {"y": y}
