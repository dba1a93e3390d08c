"""Plain 64-bit forms of the grouped products, their weight gradient and the
MX formats, and the error bounds that the GPU tests hold the kernels to.

Bounds.  A product of two operands of at most 12 significant bits is exact in
fp32; the matrix core adds products and partial sums in an order of its own,
each addition off by at most 2^-23 of a partial sum (a full unit, so that
truncation is covered too), and no partial sum exceeds S = sum |x w|.  With R
additions the sum is off by at most R 2^-23 S.  Inside one 32-value block of an
FP8 x FP4 sum the core aligns the products to the largest and drops what lies
2^-14 below it: at most 32 products by 2^-13 of max|x| max|w| (one bit of
margin, the constant the routing-combine's tests pin on the device); FP4 x FP4
products span 2^-2 .. 36 on one grid and lose nothing.  The result is rounded
once: half a step, finfo.eps / 2 of the value, or half the smallest subnormal.
"""
import numpy as np
import torch

U = 2.0 ** -23


def clamped_ends(group_list, m, list_type):
    """End row of each group as the library reads a groupList."""
    v = np.clip(np.asarray(group_list, dtype=np.int64), 0, m)
    return np.minimum(np.maximum.accumulate(v) if list_type == 0 else np.cumsum(v), m)


def groups(group_list, m, list_type):
    ends = clamped_ends(group_list, m, list_type)
    return list(zip(np.concatenate(([0], ends[:-1])), ends))


def counts_for(rng, m, e, empty=0.3, spare=0):
    """Ragged counts of e experts over m - spare rows, some of them empty."""
    share = rng.random(e) ** 3 * (rng.random(e) >= empty)
    if share.sum() == 0:
        share[rng.integers(e)] = 1.0
    c = np.floor(share / share.sum() * (m - spare)).astype(np.int64)
    c[np.argmax(share)] += m - spare - c.sum()
    return c


def as_list(counts, list_type):
    return torch.tensor(np.cumsum(counts) if list_type == 0 else counts, dtype=torch.int64)


def half_step(y, dtype):
    fi = torch.finfo(dtype)
    return y.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def product(x, w, gl, list_type):
    """x (m,k), w (e,k,n) in fp64 -> (y, S = sum |x w|); rows outside every group are NaN."""
    m, n = x.shape[0], w.shape[2]
    y = torch.full((m, n), float("nan"), dtype=torch.float64)
    s = torch.zeros((m, n), dtype=torch.float64)
    for g, (a, b) in enumerate(groups(gl, m, list_type)):
        if b > a:
            y[a:b] = x[a:b] @ w[g]
            s[a:b] = x[a:b].abs() @ w[g].abs()
    return y, s


def swiglu(y, err):
    """SwiGLU of a product known to +-err, and the bound of its own error before
    the last rounding: |silu'| <= 1.1, and the fp32 evaluation (exp of an
    argument rounded to 2^-24 |u|, a sum, a quotient, a product: under
    (8 + |u|) 2^-23 of the result)."""
    n = y.shape[1] // 2
    u, v, du, dv = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
    silu = u * torch.sigmoid(u)
    z = silu * v
    return z, 1.1 * du * (v.abs() + dv) + silu.abs() * dv + (8 + u.abs()) * U * z.abs()


def wgrad(x, dy, gl, list_type):
    e = len(gl)
    dw = torch.zeros((e, x.shape[1], dy.shape[1]), dtype=torch.float64)
    s, rows = torch.zeros_like(dw), torch.zeros(e, dtype=torch.float64)
    for g, (a, b) in enumerate(groups(gl, x.shape[0], list_type)):
        if b > a:
            dw[g] = x[a:b].T @ dy[a:b]
            s[g] = x[a:b].abs().T @ dy[a:b].abs()
            rows[g] = b - a
    return dw, s, rows


# ---------------------------------------------------------------- MX formats

FP4 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def fp8_table():
    b = np.arange(256)
    e, f, s = (b >> 3) & 15, b & 7, np.where(b >> 7, -1.0, 1.0)
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e.astype(float) - 7))
    v = np.where((b & 127) == 127, np.nan, v)
    return s * v


FP8 = fp8_table()


def elements(codes):
    """(..., k) fp64 element values of packed codes (torch CPU tensor)."""
    b = codes.view(torch.uint8).numpy()
    if codes.dtype == torch.float8_e4m3fn:
        return FP8[b]
    return np.stack((FP4[b & 15], FP4[b >> 4]), -1).reshape(*b.shape[:-1], -1)


def scale_values(scales):
    b = scales.view(torch.uint8).numpy().astype(np.float64)
    return np.where(b == 255, np.nan, 2.0 ** (b - 127)).reshape(*b.shape[:-2], -1)


def decode(codes, scales):
    v, s = elements(codes), scale_values(scales)
    return torch.from_numpy((v.reshape(*s.shape, 32) * s[..., None]).reshape(v.shape))


def encode(x, fmt):
    """(codes uint8 one per value, scales uint8) of x (..., k), fp32 numpy, by
    nearest element of the format's table, ties to the even code."""
    shape = x.shape
    x = np.asarray(x, dtype=np.float64).reshape(*shape[:-1], -1, 32)
    table = (FP4 if fmt == "fp4" else FP8)[: 8 if fmt == "fp4" else 127]
    emax = 2 if fmt == "fp4" else 8
    top = np.abs(x).max(-1)
    bad = ~np.isfinite(top)
    with np.errstate(divide="ignore", invalid="ignore"):
        s = np.where(top > 0, np.frexp(np.where(bad, 1.0, top))[1] - 1 - emax, -127)
    s = np.clip(s, -127, 127)
    v = np.where(bad[..., None], 0.0, x) * 2.0 ** -s[..., None].astype(np.float64)
    a = np.minimum(np.abs(v), table[-1])
    hi = np.clip(np.searchsorted(table, a, side="left"), 0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - table[lo], table[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(table[hi] == a, hi, code)
    sign = np.signbit(v) & ~bad[..., None]
    code = code + np.where(sign, 8 if fmt == "fp4" else 128, 0)
    return code.reshape(shape).astype(np.uint8), np.where(bad, 255, s + 127).astype(np.uint8)


def pack(code, scale, fmt):
    """Torch tensors in the library's layout from encode()'s output."""
    c = torch.from_numpy(np.ascontiguousarray(code[..., 0::2] | code[..., 1::2] << 4 if fmt == "fp4" else code))
    s = torch.from_numpy(np.ascontiguousarray(scale.reshape(*scale.shape[:-1], -1, 2)))
    return (c.view(torch.float4_e2m1fn_x2 if fmt == "fp4" else torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu))


def mx_block_loss(x_el, xs, w_el, ws):
    """FP8 x FP4: sum over blocks of 32 * 2^-13 * max|x block| max|w block|, (rows, columns)."""
    xm = np.abs(x_el.reshape(*xs.shape, 32)).max(-1) * xs
    wm = np.abs(w_el.reshape(*ws.shape, 32)).max(-1) * ws
    return torch.from_numpy(32 * 2.0 ** -13 * (xm @ wm.T))


def assert_within(got, want, bound, what=""):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {i}: "
                             f"{float(got[i])} against {float(want[i])} +- {float(bound[i])}")
