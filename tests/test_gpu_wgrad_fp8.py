"""The weight gradient of rows kept in FP8: to the bit the 16-bit one on the
widened rows, and within its bound of the 64-bit form."""
import numpy as np
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _rows(rng, m, k, wild=False):
    """FP8 rows on the host: values with blocks of unlike size, or (wild) any code but NaN under scales from 2^-40 to 2^40."""
    if wild:
        codes = rng.integers(0, 256, (m, k)).astype(np.uint8)
        codes[(codes & 127) == 127] = 0
        scales = rng.integers(87, 168, (m, k // 32)).astype(np.uint8)
        return R.pack(codes, scales, "fp8")
    x = rng.standard_normal((m, k)) * np.exp(rng.standard_normal((1, k)))
    return R.pack(*R.encode(x.astype(np.float32), "fp8"), "fp8")


def _call(codes, scale, other, gl, side, **kw):
    if side == "x":
        return B.grouped_matmul_wgrad(codes, other, gl, x_scale=scale, **kw)
    return B.grouped_matmul_wgrad(other, codes, gl, dy_scale=scale, **kw)


def _widened(values, other, gl, side, **kw):
    return B.grouped_matmul_wgrad(*((values, other) if side == "x" else (other, values)), gl, **kw)


def _case(seed, m, e, k, n, dtype, out_dtype, side, list_type, spare, tuning=None, empty=0.3, wild=False):
    """k: the columns of the FP8 rows."""
    rng = np.random.default_rng(seed)
    counts = R.counts_for(rng, m, e, empty, spare)
    end = int(counts.sum())
    gl = R.as_list(counts, list_type)
    codes, scale = _rows(rng, m, k, wild)
    dy = torch.from_numpy(rng.standard_normal((m, n)) * 0.1).to(dtype)
    scale.view(torch.uint8)[end:] = 255  # what lies behind the last group is not read
    codes.view(torch.uint8)[end:] = 127
    dy[end:] = float("nan")
    c, s, d, g = codes.cuda(), scale.cuda(), dy.cuda(), gl.cuda()
    kw = dict(group_list_type=list_type, out_dtype=out_dtype, tuning_config=tuning)
    got = _call(c, s, d, g, side, **kw)
    values = B.mx_dequantize(c, s, dtype=dtype)
    assert torch.equal(got, _widened(values, d, g, side, **kw))
    x = R.decode(codes, scale)
    if dtype == F16:  # brought to fp16 first, which rounds what it cannot hold
        x = x.to(F16).double()
    want, size, rows = R.wgrad(*((x, dy.double()) if side == "x" else (dy.double(), x)), gl.numpy(), list_type)
    bound = size * (rows + 1)[:, None, None] * R.U
    R.assert_within(got, want, bound + R.half_step(want.abs() + bound, got.dtype), "dw")
    return got


@pytest.mark.parametrize("height", [128, 256])
@pytest.mark.parametrize("side", ["x", "dy"])
@pytest.mark.parametrize("m,e,k,n,dtype,out_dtype,list_type,spare", [
    (301, 5, 320, 336, BF16, F32, 0, 7),
    (517, 3, 64, 528, F16, F16, 1, 0),
    (97, 9, 1088, 80, BF16, BF16, 1, 3),
    (33, 2, 192, 8, F16, F32, 0, 1),
    (1, 1, 64, 16, BF16, F32, 1, 0),
    (900, 4, 448, 264, BF16, F32, 1, 11),
])
def test_against_the_widened_rows(height, side, m, e, k, n, dtype, out_dtype, list_type, spare):
    _case(7, m, e, k, n, dtype, out_dtype, side, list_type, spare, tuning=[0, height])


@pytest.mark.parametrize("height", [128, 256])
@pytest.mark.parametrize("side", ["x", "dy"])
@pytest.mark.parametrize("cap", [1, 3, 16])
def test_on_few_workgroups(height, side, cap):
    """Many tiles in a row, of groups that begin at odd rows: rows of 2 scales
    modulo 4, whose bytes begin at either half of a dword."""
    for k in (320, 576, 512):
        _case(k, 611, 7, k, 392, BF16, F32, side, 1, 5, tuning=[0, height, cap])


@pytest.mark.parametrize("height", [128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_every_code_under_many_scales(height, dtype):
    """bf16 holds all of them; in fp16 the large become infinite, the small lose bits."""
    rng = np.random.default_rng(5)
    m, k, n = 290, 256, 48
    codes, scale = _rows(rng, m, k, wild=True)
    pick = torch.zeros((m, n), dtype=dtype)
    gl = torch.tensor([m]).cuda()
    for start in range(0, m, n):  # row by row: a one picks each, so sums are single values
        rows = min(n, m - start)
        pick.zero_()
        pick[start:start + rows, :rows] = torch.eye(rows, dtype=dtype)
        values = R.decode(codes, scale).to(dtype)
        if dtype == F16:  # infinity times zero
            values = torch.where(torch.isinf(values), torch.zeros_like(values), values)
            c = torch.where(torch.isinf(R.decode(codes, scale).to(dtype)), torch.zeros_like(codes.view(torch.uint8)), codes.view(torch.uint8))
            codes = c.view(torch.float8_e4m3fn)
        dw = B.grouped_matmul_wgrad(codes.cuda(), pick.cuda(), gl, x_scale=scale.cuda(), tuning_config=[0, height])
        assert torch.equal(dw[0, :, :rows].cpu(), values[start:start + rows].T.float())


@pytest.mark.parametrize("side", ["x", "dy"])
@pytest.mark.parametrize("height", [128, 256])
def test_nan_scales_stay_in_their_columns(height, side):
    rng = np.random.default_rng(6)
    m, e, k, n = 200, 2, 320, 64
    codes, scale = _rows(rng, m, k)
    scale.view(torch.uint8)[30, 2, 1] = 255   # columns 160..191 of the first group
    scale.view(torch.uint8)[150, 4, 0] = 255  # columns 256..287 of the second
    other = torch.from_numpy(rng.standard_normal((m, n))).bfloat16()
    dw = _call(codes.cuda(), scale.cuda(), other.cuda(), torch.tensor([100, 100]).cuda(), side, group_list_type=1,
               tuning_config=[0, height]).cpu()
    dw = dw if side == "x" else dw.transpose(1, 2)
    bad = torch.zeros((e, k, n), dtype=torch.bool)
    bad[0, 160:192] = True
    bad[1, 256:288] = True
    assert torch.equal(torch.isnan(dw), bad)


@pytest.mark.parametrize("side", ["x", "dy"])
def test_accumulate_and_empty(side):
    rng = np.random.default_rng(7)
    m, k, n = 150, 192, 136
    codes, scale = _rows(rng, m, k)
    other = torch.from_numpy(rng.standard_normal((m, n))).bfloat16().cuda()
    c, s = codes.cuda(), scale.cuda()
    gl = torch.tensor([70, 0, 80]).cuda()
    for height in (128, 256):
        once = _call(c, s, other, gl, side, group_list_type=1, tuning_config=[0, height])
        assert (once[1] == 0).all()
        before = torch.randn(once.shape, device="cuda")
        twice = _call(c, s, other, gl, side, out=before.clone(), accumulate=True, group_list_type=1, tuning_config=[0, height])
        assert torch.equal(twice, before + once)
        nothing = _call(c, s, other, torch.zeros_like(gl), side, group_list_type=1, tuning_config=[0, height])
        assert (nothing == 0).all()
    none = _call(c[:0], s[:0], other[:0], torch.zeros_like(gl), side)
    assert none.shape == once.shape and (none == 0).all()


@pytest.mark.parametrize("list_type,gl", [(0, [50, 30, 90]), (0, [-5, 40, 500]), (1, [30, -9, 60]), (1, [60, 60, 60])])
@pytest.mark.parametrize("height", [128, 256])
def test_broken_group_lists(list_type, gl, height):
    rng = np.random.default_rng(8)
    codes, scale = _rows(rng, 100, 64)
    dy = torch.from_numpy(rng.standard_normal((100, 72))).bfloat16()
    kw = dict(group_list_type=list_type, tuning_config=[0, height])
    got = B.grouped_matmul_wgrad(codes.cuda(), dy.cuda(), torch.tensor(gl).cuda(), x_scale=scale.cuda(), **kw)
    want, size, rows = R.wgrad(R.decode(codes, scale), dy.double(), gl, list_type)
    bound = size * (rows + 1)[:, None, None] * R.U
    R.assert_within(got, want, bound + R.half_step(want.abs() + bound, F32), "dw")


@pytest.mark.parametrize("seed", range(40))
def test_drawn(seed):
    rng = np.random.default_rng(5000 + seed)
    m, e = int(rng.integers(1, 1200)), int(rng.integers(1, 24))
    k, n = 64 * int(rng.integers(1, 14)), 8 * int(rng.integers(1, 90))
    dtype = [BF16, F16][rng.integers(2)]
    _case(seed, m, e, k, n, dtype, [dtype, F32][rng.integers(2)], ["x", "dy"][rng.integers(2)], int(rng.integers(2)),
          int(rng.integers(0, min(m, 9))), tuning=[0, int(rng.choice([0, 128, 256])), int(rng.choice([0, 0, 5, 40]))])


def test_as_many_experts_as_allowed():
    for height in (128, 256):
        for side in ("x", "dy"):
            _case(23, 3000, 1024, 64, 40, BF16, F32, side, 1, 2, tuning=[0, height], empty=0.4)
