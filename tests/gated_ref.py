"""Plain 64-bit forms of the gated feed-forward block and of its way back, and
the error bounds that the GPU tests hold the kernels to.

  h = a(u) v,  a(u) = u s(z),  s(z) = 1 / (1 + exp(-z));
  silu: z = u, gelu: z = sqrt(8/pi) (u + 0.044715 u^3)
  du = dh v a'(u),  a'(u) = s + u z'(u) s (1 - s),  dv = dh a(u)

Bounds.  Sums are off by (terms + 1) 2^-23 sum |x w|, as in grouped_ref.  The
gate in fp32: z (its constants rounded, a square, a fused product and a product)
is off by 5 2^-24 |z| at most, so exp(-z), and s and 1 - s with it, by that much
of themselves, and by 4 2^-23 from exp, sum and reciprocal (1 ulp each, and the
rounding of exp's argument counted above); each further product or sum adds half
of 2^-23.  (8 + 3 |z|) 2^-23 of the result covers the values, and the same of
|s| + |u z' s (1 - s)|, whose sum may cancel, with two more products, the
derivative.  |silu'| < 1.1 and |gelu'| < 1.13, so an error of u becomes at most
1.13 times that of a(u).
"""
import math

import torch

from tests import grouped_ref as R

C = math.sqrt(8 / math.pi)


def gate(u, act):
    """z, a(u), a'(u) and |s| + |u z' s (1 - s)|, in fp64 and without overflow."""
    if act == "swiglu":
        z, slope = u, torch.ones_like(u)
    else:
        z, slope = C * (u + 0.044715 * u ** 3), C * (1 + 3 * 0.044715 * u * u)
    s, rest = torch.sigmoid(z), torch.sigmoid(-z)
    bend = u * slope * s * rest
    return z, u * s, s + bend, s + bend.abs()


def forward(both, err, act):
    """h of projections (u | v) known to +-err, and its bound before the rounding."""
    f = both.shape[1] // 2
    u, v, du, dv = both[:, :f], both[:, f:], err[:, :f], err[:, f:]
    z, a, _, _ = gate(u, act)
    h = a * v
    return h, 1.13 * du * (v.abs() + dv) + a.abs() * dv + (8 + 3 * z.abs()) * R.U * h.abs()


def backward(dh, err, both, act):
    """(du | dv) and h of dh known to +-err and of exact u and v; their bounds before the rounding."""
    f = both.shape[1] // 2
    u, v = both[:, :f], both[:, f:]
    z, a, slope, size = gate(u, act)
    own = (8 + 3 * z.abs()) * R.U
    d = torch.cat((dh * v * slope, dh * a), 1)
    bound = torch.cat((err * (v * slope).abs() + (own + R.U) * ((dh.abs() + err) * v.abs() * size),
                       err * a.abs() + own * (dh.abs() + err) * a.abs()), 1)
    h = a * v
    return d, bound, h, own * h.abs()


def fp8_bound(y, err):
    """How far the values that E4M3 codes with a scale per 32 stand for may be
    from y, itself known to +-err: half a step of the format (2^-4 of the value,
    or 2^-10 of the scale, whose exponent follows the largest value), and what a
    value past 448 of the scale loses, for either exponent that err allows."""
    blocks = y.abs().unflatten(1, (-1, 32))
    e = err.unflatten(1, (-1, 32))
    high = (blocks + e).amax(-1, keepdim=True).clamp(min=2.0 ** -118)
    low = (blocks - e).amax(-1, keepdim=True).clamp(min=2.0 ** -118)
    s_high, s_low = 2.0 ** (torch.floor(torch.log2(high)) - 8), 2.0 ** (torch.floor(torch.log2(low)) - 8)
    half = torch.maximum((blocks + e) * 2.0 ** -4, s_high * 2.0 ** -10)
    return (e + half + (blocks + e - 448 * s_low).clamp(min=0)).flatten(1)
