"""More of the grouped products: a weight gradient against differences within a
bound that a missing row exceeds, broken group lists through the weight
gradient and the microscaled products, expected rows, and repeated calls."""
import numpy as np
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import grouped_ref as R
from tests import test_gpu_grouped as T

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = 7.25


@pytest.mark.parametrize("height", [128, 256])
def test_wgrad_against_differences_of_its_own_column(height):
    """dw[g,p,j] against (Y(+) - Y(-)) / (w(+) - w(-)) with Y = sum over the
    group's rows of dy[i,j] y[i,j], the library's product in fp32.  Y is linear
    in w[g,p,j]: the quotient is off only by y's own error, at most (k + 2)
    2^-23 of S_i = sum_q |x_iq| |w_qj| in each of the two (the k + 1 additions
    and the rounding to fp32), and dw by (rows + 2) 2^-23 of sum |x dy|.  The
    bound has to be below what the largest row's term is worth."""
    rng = np.random.default_rng(25)
    m, e, k, n = 90, 3, 40, 48
    counts = [50, 0, 40]
    gl = torch.tensor(counts)
    x, w = T._rand(rng, (m, k), BF16), T._rand(rng, (e, k, n), BF16)
    dy = T._rand(rng, (m, n), BF16)
    dw = B.grouped_matmul_wgrad(x.cuda(), dy.cuda(), gl.cuda(), group_list_type=1, tuning_config=[0, height]).cpu().double()
    xd, dyd = x.double(), dy.double()
    for g, p, j in [(0, 0, 0), (0, 39, 47), (0, 17, 31), (2, 17, 20), (2, 0, 47), (2, 39, 8)]:
        a = sum(counts[:g])
        rows = slice(a, a + counts[g])
        moved, total, s = [], [], 0.0
        for sign in (1, -1):
            v = w.clone()
            v[g, p, j] = float(w[g, p, j]) + 0.5 * sign
            moved.append(float(v[g, p, j]))
            y = B.grouped_matmul(x.cuda(), v.cuda(), gl.cuda(), out_dtype=F32, group_list_type=1).cpu().double()
            total.append(float((dyd[rows, j] * y[rows, j]).sum()))
            s += float((dyd[rows, j].abs() * (xd[rows].abs() @ v[g, :, j].double().abs())).sum())
        step = moved[0] - moved[1]
        term = (xd[rows, p] * dyd[rows, j]).abs()
        bound = s * (k + 2) * R.U / step + float(term.sum()) * (counts[g] + 2) * R.U
        assert abs((total[0] - total[1]) / step - float(dw[g, p, j])) <= bound, (g, p, j)
        assert bound < 0.05 * float(term.max()), (g, p, j)  # a gradient without that row would not pass


BROKEN = [(0, [40, 10, 90, 500]), (1, [30, -5, 60, 10 ** 12]), (0, [-7, 120, 3, 10 ** 18]), (1, [200, 1, -(10 ** 15), 4])]


@pytest.mark.parametrize("height", [128, 256])
@pytest.mark.parametrize("list_type,gl", BROKEN)
def test_broken_group_lists_of_the_weight_gradient(list_type, gl, height):
    rng = np.random.default_rng(26)
    m, e, k, n = 120, 4, 72, 88
    x, dy = T._rand(rng, (m, k), BF16), T._rand(rng, (m, n), BF16)
    want, s, rows = R.wgrad(x.double(), dy.double(), np.array(gl), list_type)
    bound = s * (rows + 1)[:, None, None] * R.U
    big = torch.full((e + 2, k, n), SENTINEL, dtype=F32, device="cuda")
    for accumulate in (False, True):
        big.fill_(SENTINEL)
        B.grouped_matmul_wgrad(x.cuda(), dy.cuda(), torch.tensor(gl).cuda(), out=big[1:1 + e], group_list_type=list_type,
                               accumulate=accumulate, tuning_config=[0, height])
        total = want + SENTINEL if accumulate else want
        R.assert_within(big[1:1 + e], total, bound + R.half_step(total.abs() + bound, F32), f"accumulate {accumulate}")
        assert (big[0] == SENTINEL).all() and (big[-1] == SENTINEL).all()


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("list_type,gl", BROKEN)
def test_broken_group_lists_of_microscaled_products(list_type, gl, fmt, height):
    rng = np.random.default_rng(27)
    m, e, k, n = 120, 4, 192, 80
    x, xs = T._mx_operand(rng, (m, k), fmt)
    w, ws = T._mx_operand(rng, (e, n, k), "fp4", k ** -0.5)
    want, s = R.product(R.decode(x, xs), R.decode(w, ws).transpose(1, 2), np.array(gl), list_type)
    err = s * (k // 32 + 32) * R.U
    if fmt == "fp8":
        xe, xv, we, wv = R.elements(x), R.scale_values(xs), R.elements(w), R.scale_values(ws)
        for g, (a, b) in enumerate(R.groups(gl, m, list_type)):
            if b > a:
                err[a:b] += R.mx_block_loss(xe[a:b], xv[a:b], we[g], wv[g])
    big = torch.full((m + 64, n), SENTINEL, dtype=F32, device="cuda")
    B.grouped_matmul(x.cuda(), w.cuda(), torch.tensor(gl).cuda(), x_scale=xs.cuda(), w_scale=ws.cuda(), out=big[32:32 + m],
                     transpose_w=True, group_list_type=list_type, tuning_config=[0, height])
    end = int(R.clamped_ends(gl, m, list_type)[-1])
    assert (big[:32] == SENTINEL).all() and (big[32 + end:] == SENTINEL).all()
    R.assert_within(big[32:32 + end], want[:end], (err + R.half_step(want.abs() + err, F32))[:end], "product")


@pytest.mark.parametrize("rows", [1, 20, 100, 1000, 2 ** 62])
def test_expected_rows(rows):
    """Whatever is expected, the product is right."""
    T._dense_case(28, 700, 6, 136, 648, BF16, BF16, False, None, 1, 5, tuning=[rows])
    T._dense_case(29, 90, 40, 136, 272, F16, F32, True, "swiglu", 0, 1, tuning=[rows])
    T._mx_case(30, 500, 6, 320, 400, "fp8", F32, None, 1, 5, tuning=[rows])
    T._mx_case(31, 500, 6, 320, 400, "fp4", BF16, "swiglu", 0, 5, tuning=[rows])


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_microscaled_calls_repeat_themselves(fmt, height):
    """Bit for bit, whatever the grid: the sums have one order."""
    rng = np.random.default_rng(32)
    m, e, k, n = 900, 5, 1088, 400
    gl = R.as_list(R.counts_for(rng, m, e), 1).cuda()
    (x, xs), (w, ws) = T._mx_operand(rng, (m, k), fmt), T._mx_operand(rng, (e, n, k), "fp4")
    x, xs, w, ws = x.cuda(), xs.cuda(), w.cuda(), ws.cuda()

    def call(cap):
        return B.grouped_matmul(x, w, gl, x_scale=xs, w_scale=ws, transpose_w=True, group_list_type=1, out_dtype=F32,
                                tuning_config=[0, height, cap])
    first = call(0)
    for cap in (0, 0, 1, 7, 64):
        assert torch.equal(first, call(cap)), cap
