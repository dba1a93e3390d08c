"""The gate of the gated block, forward and back, for gates of every size, large
positive ones among them, within a few units of fp32 of the 64-bit value.

Bounds, in units of U = 2^-23 (exp2 and the reciprocal within one, a rounding half
of one), with s = 1 / (1 + e), e = exp(-z) and dh exact:
  - z's constants, square, fused product and product are off by 3 |z| of it, so e
    by 3 |z| + 1; s by (1 - s) of that, as d(log s) = (1 - s) d(log e), and by 1.5.
  - a = u s and each product with it add 0.5: a v and dh a are within
    4 + 3 |z| (1 - s) of themselves.  Past z = 0 the second part dies out.
  - a' = s + bend, bend = u z' s (1 - s): e s, from the same e, is off by
    s (3 |z| + 1) + 2, z' by 2, a by the above, three products and their sum: the
    bend by 3 |z| + 9 of itself, the rest by 5 + 3 |z| (1 - s) of s.
  - Below z = -87 s is exp(z / 2) twice, each off by 1.5 |z| + 1 (half the
    exponent), with up to four products: within the same.
fp32 flushes what is below 2^-126.
"""
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import gated_ref as G
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
FLOOR = 2.0 ** -126
SIZES = [0.0, 1e-30, 1e-6, 0.3, 1.0, 1.2785, 3.0, 5.5, 9.0, 9.98, 10.0, 10.2, 11.0, 12.5, 15.9, 16.1, 17.0, 30.0, 60.0, 80.0, 86.0,
         87.0, 87.25, 87.5, 88.0, 88.75, 90.0, 100.0, 120.0, 170.0, 1e3, 6e4]


def _parts(u, act):
    """z, a(u), s, 1 - s and the bend u z' s (1 - s), in fp64 and without overflow."""
    if act == "swiglu":
        z, slope = u, torch.ones_like(u)
    else:
        z, slope = G.C * (u + 0.044715 * u ** 3), G.C * (1 + 3 * 0.044715 * u * u)
    s, rest = torch.sigmoid(z), torch.sigmoid(-z)
    return z, u * s, s, rest, u * slope * s * rest


def _forward(u, v, act):
    z, a, _, rest, _ = _parts(u, act)
    return a * v, (4 + 3 * z.abs() * rest) * R.U * (a * v).abs()


def _backward(dh, u, v, act):
    z, a, s, rest, bend = _parts(u, act)
    own = (4 + 3 * z.abs() * rest) * R.U
    slope = ((9 + 3 * z.abs()) * bend.abs() + (5 + 3 * z.abs() * rest) * s) * R.U
    return (torch.cat((dh * v * (s + bend), dh * a), 1), torch.cat((dh * v.abs() * slope, own * (dh * a).abs()), 1).abs(),
            a * v, own * (a * v).abs())


def _check(got, want, bound, what):
    """Where the result fits the type: what passes its range is not compared."""
    fits = want.abs() < torch.finfo(got.dtype).max * (1 - 2.0 ** -7)
    R.assert_within(torch.where(fits, got.cpu().double(), want), want, bound + R.half_step(want, got.dtype) + FLOOR, what)


def _gates(dtype, sizes):
    g = torch.tensor(sizes, dtype=torch.float64)
    g = torch.cat((g, -g, torch.ones(-2 * len(g) % 8, dtype=torch.float64)))  # whole chunks of 8
    return g.to(dtype)


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_forward(dtype, height, act):
    """One row of x picks one row of w, so that the sums are the weights."""
    g = _gates(dtype, SIZES + ([1e10, 1e30] if dtype == BF16 else []))
    up = torch.tensor([1.0, -2.0 ** 14, 2.0 ** -14, 2.0 ** 100 if dtype == BF16 else 3.0]).to(dtype)
    m, f = len(up), len(g)
    both = torch.cat((g.expand(m, f), up[:, None].expand(m, f)), 1)
    x, w = torch.zeros((m, 8), dtype=dtype), torch.zeros((1, 8, 2 * f), dtype=dtype)
    x[:, :m], w[0, :m] = torch.eye(m, dtype=dtype), both
    h, _, _ = B.gated_matmul(x.cuda(), w.cuda(), torch.tensor([m]).cuda(), activation=act, tuning_config=[0, height])
    u, v = both.double().chunk(2, 1)
    _check(h, *_forward(u, v, act), "h")


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("keep,dtype", [("full", BF16), ("full", F16), ("fp8", BF16)])
def test_backward(keep, dtype, height, act):
    """dh is dy where the weights are one.  Kept in FP8 every gate is a block of its own."""
    g = _gates(dtype, SIZES + ([1e10, 1e30] if dtype == BF16 else []))
    up = torch.tensor([1.0, -2.0 ** 14, 2.0 ** -14, 2.0 ** 100 if dtype == BF16 else 3.0]).to(dtype)
    if keep == "fp8":
        g = g.repeat_interleave(32)
    m, f = len(up), len(g)
    kept, scale = torch.cat((g.expand(m, f), up[:, None].expand(m, f)), 1).contiguous().cuda(), None
    if keep == "fp8":
        kept, scale = B.mx_quantize(kept, format="fp8")
    u, v = (kept.cpu().double() if scale is None else R.decode(kept.cpu(), scale.cpu())).chunk(2, 1)
    ones = torch.ones((1, f, 8), dtype=dtype, device="cuda")
    for dh in (1.0, 2.0 ** -10, -2.0 ** 5):
        dy = torch.zeros((m, 8), dtype=dtype, device="cuda")
        dy[:, 0] = dh
        d, h = B.gated_matmul_backward(dy, ones, torch.tensor([m]).cuda(), kept, kept_scale=scale, activation=act, tuning_config=[0, height])
        want, bound, h_want, h_bound = _backward(torch.full((m, f), dh, dtype=torch.float64), u, v, act)
        _check(d, want, bound, f"gradients, dh = {dh}")
        _check(h, h_want, h_bound, f"h again, dh = {dh}")


HUGE = [6e36, 6.2e36, 1e37, 1e38, 3.3e38]  # z' u passes fp32's range from 6.1e36 on


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("keep", ["full", "fp8"])
def test_gates_up_to_the_largest(keep, height, act):
    """du is dh v behind a large positive gate, 0 behind a large negative one."""
    g = _gates(BF16, [*HUGE, 1.0])
    if keep == "fp8":
        g = g.repeat_interleave(32)
    up = torch.tensor([1.0, -2.0 ** -14, 2.0 ** -20, 1.5]).to(BF16)
    m, f = len(up), len(g)
    both = torch.cat((g.expand(m, f), up[:, None].expand(m, f)), 1).contiguous()
    x, w = torch.zeros((m, 8), dtype=BF16), torch.zeros((1, 8, 2 * f), dtype=BF16)
    x[:, :m], w[0, :m] = torch.eye(m, dtype=BF16), both
    gl, tuning = torch.tensor([m]).cuda(), [0, height]
    h, kept, scale = B.gated_matmul(x.cuda(), w.cuda(), gl, keep=keep, activation=act, tuning_config=tuning)
    u, v = both.double().chunk(2, 1)
    _check(h, *_forward(u, v, act), "h")
    u, v = (kept.cpu().double() if scale is None else R.decode(kept.cpu(), scale.cpu())).chunk(2, 1)
    dy = torch.zeros((m, 8), dtype=BF16, device="cuda")
    dy[:, 0] = 2.0 ** -3
    d, h = B.gated_matmul_backward(dy, torch.ones((1, f, 8), dtype=BF16, device="cuda"), gl, kept, kept_scale=scale, activation=act,
                                   tuning_config=tuning)
    want, bound, h_want, h_bound = _backward(torch.full((m, f), 2.0 ** -3, dtype=torch.float64), u, v, act)
    _check(d, want, bound, "gradients")
    _check(h, h_want, h_bound, "h again")
