"""The grouped products, the weight gradient and the MX quantisation at the
largest k and n they take, sampled against 64-bit forms within grouped_ref's
bounds.  Those are worst cases, wide for sums this long: the sampled outputs as
a whole also stay within 2^-13 of their norm (fp32) or 2^-8 (bf16)."""
import numpy as np
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
MOST = 65536


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _normal(seed, *shape, dtype=BF16, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=dtype, device="cuda")
    for part in t.view(-1).split(2 ** 30):
        part.normal_(0, scale, generator=gen)
    return t


def _bytes(seed, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for part in t.view(-1).split(2 ** 30):
        part.random_(0, 256, generator=gen)
    return t


def _columns(n):
    return sorted({c for c in (0, 1, 31, 32, 63, 255, 256, n // 2 - 1, n // 2, n - 257, n - 8, n - 1) if 0 <= c < n})


def _close(y, want, err, dtype):
    R.assert_within(y, want, err + R.half_step(want.abs() + err, dtype))
    assert float((y.double() - want).norm() / want.norm()) <= (2.0 ** -13 if dtype == F32 else 2.0 ** -8)


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("k,n,act", [(MOST, 16, None), (8, MOST, None), (MOST, MOST, None), (MOST, 16384, "swiglu"),
                                     (16384, MOST, "swiglu")])
def test_16_bit_products(height, transpose, k, n, act):
    """(65536, 16384) and (16384, 65536) with SwiGLU: an expert's weights of just 2 GiB."""
    m, out = 5, F32 if k == MOST else BF16
    x = _normal(1, m, k)
    w = _normal(2, 1, *((n, k) if transpose else (k, n)), scale=k ** -0.5)
    y = B.grouped_matmul(x, w, torch.tensor([m], device="cuda"), transpose_w=transpose, activation=act, out_dtype=out,
                         tuning_config=[0, height]).cpu()
    half = n // 2 if act else n
    cols = _columns(half)

    def some(c):
        c = torch.tensor(c, device="cuda")
        return (w[0].index_select(0, c).T if transpose else w[0].index_select(1, c)).cpu().double()
    both = some(cols + [c + half for c in cols]) if act else some(cols)
    xd = x.cpu().double()
    want, err = xd @ both, xd.abs() @ both.abs() * (k + 1) * R.U
    if act:
        want, err = R.swiglu(want, err)
    _close(y[:, cols], want, err, out)


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("k,n,act", [(MOST, 16, None), (64, MOST, None), (MOST, MOST, "swiglu")])
def test_microscaled_products(height, fmt, k, n, act):
    m = 5
    x = _normal(3, m, k)
    xc, xs = B.mx_quantize(x, format=fmt)
    wb = _bytes(4, 1, n, k // 2)
    ws = (_bytes(5, 1, n, k // 64, 2) % 8 + 112)
    y = B.grouped_matmul(xc, wb.view(torch.float4_e2m1fn_x2), torch.tensor([m], device="cuda"), x_scale=xs,
                         w_scale=ws.view(torch.float8_e8m0fnu), transpose_w=True, activation=act, out_dtype=F32,
                         tuning_config=[0, height]).cpu()
    half = n // 2 if act else n
    cols = _columns(half)
    at = cols + [c + half for c in cols] if act else cols
    pick = torch.tensor(at, device="cuda")
    wc = wb[0].index_select(0, pick).cpu().view(torch.float4_e2m1fn_x2)
    wsc = ws[0].index_select(0, pick).cpu().view(torch.float8_e8m0fnu)
    xd, wd = R.decode(xc.cpu(), xs.cpu()), R.decode(wc, wsc)
    want, err = xd @ wd.T, xd.abs() @ wd.abs().T * (k // 32 + 32) * R.U
    if fmt == "fp8":
        err = err + R.mx_block_loss(R.elements(xc.cpu()), R.scale_values(xs.cpu()), R.elements(wc), R.scale_values(wsc))
    if act:
        want, err = R.swiglu(want, err)
    _close(y[:, cols], want, err, F32)


@pytest.mark.parametrize("height", [128, 256])
@pytest.mark.parametrize("k,n", [(MOST, MOST), (8, MOST), (MOST, 8)])
def test_weight_gradient(height, k, n):
    m = 70
    x, dy = _normal(6, m, k), _normal(7, m, n)
    dw = B.grouped_matmul_wgrad(x, dy, torch.tensor([m], device="cuda"), tuning_config=[0, height])
    rows, cols = _columns(k), _columns(n)
    xd, dyd = x[:, rows].cpu().double(), dy[:, cols].cpu().double()
    got = dw[0].index_select(0, torch.tensor(rows, device="cuda")).index_select(1, torch.tensor(cols, device="cuda")).cpu()
    _close(got, xd.T @ dyd, xd.abs().T @ dyd.abs() * (m + 1) * R.U, F32)


@pytest.mark.parametrize("height", [32, 128, 256])
def test_microscaled_weights_past_32_bits(height):
    """Nine gigabytes of FP4 weights, rows in the first, a middle and the last expert."""
    e, n, k = 600, 4096, 7168
    counts = torch.zeros(e, dtype=torch.int64)
    counts[0], counts[311], counts[599] = 2, 3, 4
    x = _normal(8, 9, k)
    xc, xs = B.mx_quantize(x)
    wb, ws = _bytes(9, e, n, k // 2), _bytes(10, e, n, k // 64, 2) % 8 + 112
    y = B.grouped_matmul(xc, wb.view(torch.float4_e2m1fn_x2), counts.cuda(), x_scale=xs, w_scale=ws.view(torch.float8_e8m0fnu),
                         transpose_w=True, group_list_type=1, out_dtype=F32, tuning_config=[0, height]).cpu()
    xd, cols, first = R.decode(xc.cpu(), xs.cpu()), _columns(n), 0
    for g in (0, 311, 599):
        c = int(counts[g])
        wd = R.decode(wb[g][cols].cpu().view(torch.float4_e2m1fn_x2), ws[g][cols].cpu().view(torch.float8_e8m0fnu))
        part = xd[first:first + c]
        _close(y[first:first + c][:, cols], part @ wd.T, part.abs() @ wd.abs().T * (k // 32 + 32) * R.U, F32)
        first += c


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantisation(fmt, transpose):
    x = _normal(11, 1, MOST, 8) if transpose else _normal(11, 3, MOST)
    codes, scales = B.mx_quantize(x, format=fmt, transpose=transpose)
    v = (x.transpose(1, 2) if transpose else x).float().cpu().numpy()
    pc, ps = R.pack(*R.encode(v, fmt), fmt)
    assert torch.equal(codes.view(torch.uint8).cpu(), pc.view(torch.uint8))
    assert torch.equal(scales.view(torch.uint8).cpu(), ps.view(torch.uint8))
    assert torch.equal(B.mx_dequantize(codes, scales, dtype=F32).cpu(), R.decode(pc, ps).float())
