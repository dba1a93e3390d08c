"""SwiGLU of gates over the whole range of fp32's exponential, in the epilogue
of the grouped products, against u / (1 + exp(-u)) * v in 64 bits.

A gate and an up value are each one product by 1 among zeros, so they reach the
epilogue exactly and only the activation's own error counts: grouped_ref.swiglu
bounds it by (8 + |u|) 2^-23 of the result.  Results below fp32's normal range
are off by half the smallest subnormal for the rounding (half_step) and once
more for an intermediate below that range."""
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
GATES = [-104.0, -103.0, -96.0, -92.0, -90.0, -89.0, -88.5, -88.0, -87.5, -87.0, -80.0, -60.0, -20.0, -8.0, -2.0, -1.0,
         -0.25, -2.0 ** -20, 0.0, 2.0 ** -20, 0.25, 1.0, 2.0, 8.0, 20.0, 60.0, 87.5, 88.0, 92.0, 104.0, -120.0, -170.0,
         -1000.0, 180.0, 1000.0]
UPS = {BF16: [1.0, -0.75, 2.0 ** 60, -(2.0 ** 126), 3.0 * 2.0 ** 126, 2.0 ** -100], F16: [1.0, -0.75, 60000.0, 2.0 ** -14]}


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
def test_swiglu_over_the_gates_range(height, transpose, dtype, out_dtype):
    k, f, ups = 64, 16, UPS[dtype]
    u = torch.tensor(GATES, dtype=torch.float64).repeat_interleave(len(ups))
    v = torch.tensor(ups, dtype=torch.float64).repeat(len(GATES))
    x = torch.zeros((len(u), k), dtype=dtype)
    x[:, 3], x[:, 40] = u.to(dtype), v.to(dtype)
    u, v = x[:, 3].double(), x[:, 40].double()
    w = torch.zeros((1, k, 2 * f), dtype=dtype)
    w[0, 3, :f], w[0, 40, f:] = 1, 1
    if transpose:
        w = w.transpose(1, 2).contiguous()
    y = B.grouped_matmul(x.cuda(), w.cuda(), torch.tensor([len(u)]).cuda(), transpose_w=transpose, activation="swiglu",
                         out_dtype=out_dtype, tuning_config=[0, height])
    both = torch.cat([u[:, None].expand(-1, f), v[:, None].expand(-1, f)], 1)
    want, err = R.swiglu(both, torch.zeros_like(both))
    # out of 16 bits' range the rounding gives an infinity
    fits = (want.abs() < torch.finfo(out_dtype).max).cpu()
    bound = err + R.half_step(want.abs() + err, out_dtype) + 2.0 ** -150
    got = y.double().cpu()
    R.assert_within(torch.where(fits, got, 0.0), torch.where(fits, want, 0.0), bound, "swiglu")
    assert torch.equal(torch.isinf(got), ~fits)


@pytest.mark.parametrize("height", [32, 128, 256])
def test_swiglu_of_microscaled_gates(height):
    """The same for FP8 rows with FP4 weights, whose epilogue is the same code
    in other instances: gates of 8 E4M3 steps, ups of large block scales."""
    gates = torch.tensor([-104.0, -96.0, -88.0, -80.0, -1.0, 1.0, 88.0])
    k, f = 64, 16
    code = torch.zeros((len(gates), k))
    code[:, 3], code[:, 40] = gates, 1.0
    scale = torch.full((len(gates), 1, 2), 127, dtype=torch.uint8)
    scale[:, 0, 1] = 127 + 90  # up: 2^90
    one = torch.zeros((1, 2 * f, k // 2), dtype=torch.uint8)
    one[0, :f, 1] = 0x20   # FP4 1.0 at the odd position 3
    one[0, f:, 20] = 0x02  # and at the even position 40
    ws = torch.full((1, 2 * f, 1, 2), 127, dtype=torch.uint8)
    y = B.grouped_matmul(code.to(torch.float8_e4m3fn).cuda(), one.view(torch.float4_e2m1fn_x2).cuda(),
                         torch.tensor([len(gates)]).cuda(), x_scale=scale.view(torch.float8_e8m0fnu).cuda(),
                         w_scale=ws.view(torch.float8_e8m0fnu).cuda(), transpose_w=True, activation="swiglu", out_dtype=F32,
                         tuning_config=[0, height])
    both = torch.cat([gates.double()[:, None].expand(-1, f), torch.full((len(gates), f), 2.0 ** 90, dtype=torch.float64)], 1)
    want, err = R.swiglu(both, torch.zeros_like(both))
    R.assert_within(y, want, err + R.half_step(want.abs() + err, F32), "swiglu")


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_a_row_does_not_depend_on_its_neighbours_gates(height, out_dtype):
    """Rows beside ones with far gates, bit for bit as without them."""
    gen = torch.Generator().manual_seed(33)
    m, k, f = 96, 64, 64
    x = torch.randn((m, k), generator=gen).to(BF16)
    w = torch.randn((1, k, 2 * f), generator=gen).to(BF16)
    w[0, 0, :f] = 1
    x[:, 0] = 0
    gl = torch.tensor([m]).cuda()

    def call(x):
        return B.grouped_matmul(x.cuda(), w.cuda(), gl, activation="swiglu", out_dtype=out_dtype, tuning_config=[0, height]).cpu()
    far = torch.arange(m) % 7 == 3
    beside = x.clone()
    beside[far, 0] = -200.0
    assert torch.equal(call(x)[~far], call(beside)[~far])
