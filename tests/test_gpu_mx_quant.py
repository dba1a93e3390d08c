"""Microscaled quantisation and its inverse against a table-driven 64-bit
reading: codes, scales and values bit for bit."""
import numpy as np
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _check(x, fmt, transpose=False):
    """x: CPU tensor in its type."""
    codes, scales = B.mx_quantize(x.cuda(), format=fmt, transpose=transpose)
    v = (x.transpose(1, 2) if transpose else x).float().numpy()
    want_c, want_s = R.encode(v, fmt)
    pc, ps = R.pack(want_c, want_s, fmt)
    assert codes.shape == pc.shape and scales.shape == ps.shape
    got_s = scales.view(torch.uint8).cpu()
    assert torch.equal(got_s, ps.view(torch.uint8)), (got_s != ps.view(torch.uint8)).nonzero()[:5]
    got_c = codes.view(torch.uint8).cpu()
    assert torch.equal(got_c, pc.view(torch.uint8)), (got_c != pc.view(torch.uint8)).nonzero()[:5]
    values = R.decode(pc, ps)
    for dtype in TYPES.values():
        got = B.mx_dequantize(codes, scales, dtype=dtype).cpu()
        want = values.to(torch.float32).to(dtype)  # code * 2^s is exact in fp32 down to 2^-149
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want)), dtype


def _wide(rng, shape, spread):
    v = rng.standard_normal(shape) * np.exp2(rng.integers(-spread, spread + 1, shape[:-1])[..., None])
    return v.astype(np.float32)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 64), (3, 192), (37, 2112), (8, 7168), (2, 5, 320), (1025, 64)])
def test_rows(fmt, name, shape):
    rng = np.random.default_rng(shape[-1])
    _check(torch.from_numpy(_wide(rng, shape, 10 if name == "fp16" else 60)).to(TYPES[name]), fmt)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 64, 8), (2, 192, 136), (3, 320, 40), (1, 576, 264), (2, 256, 128)])
def test_transposed_weights(fmt, name, shape):
    rng = np.random.default_rng(shape[1])
    x = _wide(rng, (shape[0], shape[2], shape[1]), 8).transpose(0, 2, 1).copy()
    _check(torch.from_numpy(x).to(TYPES[name]), fmt, transpose=True)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("transpose", [False, True])
def test_ties_borders_and_special_blocks(fmt, transpose):
    """Half-way values, the format's largest and what saturates, zeros of both
    signs, subnormal and huge blocks, and blocks with a NaN or an infinity."""
    table = R.FP4[:8] if fmt == "fp4" else R.FP8[:127]
    top = table[-1]
    half = (table[1:] + table[:-1]) / 2
    values = np.concatenate([table, half, [top * 1.05, top * 1.15, top * 1.3 if fmt == "fp4" else top * 1.14]])
    values = np.concatenate([values, -values])
    rows = []
    for scale in (-126, -30, 0, 40, 118):
        v = np.resize(values, (len(values) + 30) // 31 * 31).reshape(-1, 31) * 2.0 ** scale
        rows.append(np.concatenate([np.full((len(v), 1), top * 2.0 ** scale), v], 1))  # pins the block's exponent
    special = np.zeros((8, 32))
    special[1] = -0.0
    special[2, 5] = 1e-40
    special[3] = np.float32(2.0 ** -149)
    special[4] = np.linspace(-3.4e38, 3.4e38, 32)
    special[5] = 1.0
    special[5, 31] = np.nan
    special[6] = -2.0
    special[6, 0] = np.inf
    special[7] = np.linspace(1, 2, 32)
    blocks = np.concatenate(rows + [special]).astype(np.float32)
    if len(blocks) % 2:
        blocks = np.concatenate([blocks, blocks[-1:]])
    x = torch.from_numpy(blocks).reshape(-1, 64)
    if transpose:
        pad = -x.shape[0] % 8
        x = torch.cat([x, x[:pad]]).T.contiguous()[None]
    _check(x, fmt, transpose)
    _check(x.bfloat16(), fmt, transpose)


@pytest.mark.parametrize("rows", [0, 1])
def test_no_and_one_row(rows):
    x = torch.ones((rows, 64), dtype=torch.bfloat16, device="cuda")
    codes, scales = B.mx_quantize(x)
    assert codes.shape == (rows, 32) and scales.shape == (rows, 1, 2)
    assert torch.equal(B.mx_dequantize(codes, scales), x)


def test_past_32_bits():
    """4.4e9 values: the last rows' codes, from a tensor that repeats a small one."""
    small = torch.randn((256, 8192), device="cuda").bfloat16()
    x = small.repeat(2100, 1)
    codes, scales = B.mx_quantize(x, format="fp8")
    c, s = B.mx_quantize(small, format="fp8")
    assert torch.equal(codes.view(torch.uint8)[-256:], c.view(torch.uint8))
    assert torch.equal(scales.view(torch.uint8)[-256:], s.view(torch.uint8))
