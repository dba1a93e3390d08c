"""Grouped products (16-bit and microscaled, plain and SwiGLU) and the weight
gradient against plain 64-bit forms, within bounds derived in grouped_ref.py."""
import numpy as np
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = 7.25


def _rand(rng, shape, dtype, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(dtype)


def _poison_outside(x, ends):
    """NaN and infinity in the rows behind the last group."""
    x[ends[-1]:] = float("nan")
    if x.shape[0] - ends[-1] > 1:
        x[ends[-1] + 1:] = float("inf")


def _check_product(y, want, bound, dtype, end, m):
    y = y.cpu()
    assert y.dtype == dtype
    R.assert_within(y[:end], want[:end], (bound + R.half_step(want.abs() + bound, dtype))[:end], "product")
    assert (y[end:] == SENTINEL).all(), "rows behind the last group were written"


def _dense_case(seed, m, e, k, n, dtype, out_dtype, transpose, act, list_type, spare, tuning=None, empty=0.3):
    rng = np.random.default_rng(seed)
    counts = R.counts_for(rng, m, e, empty, spare)
    gl = R.as_list(counts, list_type)
    x = _rand(rng, (m, k), dtype)
    w = _rand(rng, (e, n, k) if transpose else (e, k, n), dtype, k ** -0.5)
    _poison_outside(x, np.cumsum(counts))
    w[counts == 0] = float("nan")  # an expert without rows is never read
    xd = x.double()
    wd = (w.transpose(1, 2) if transpose else w).double()
    want, s = R.product(xd, wd, gl.numpy(), list_type)
    err = s * (k + 1) * R.U
    if act == "swiglu":
        want, err = R.swiglu(want, err)
    out = torch.full((m, n // 2 if act else n), SENTINEL, dtype=out_dtype, device="cuda")
    y = B.grouped_matmul(x.cuda(), w.cuda(), gl.cuda(), out=out, transpose_w=transpose, activation=act,
                         group_list_type=list_type, tuning_config=tuning)
    assert y is out
    _check_product(y, want, err, out_dtype, int(counts.sum()), m)
    return y


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("m,e,k,n,dtype,out_dtype,list_type,spare", [
    (301, 5, 264, 336, BF16, BF16, 0, 7),
    (517, 3, 72, 528, F16, F16, 1, 0),
    (97, 9, 1032, 80, BF16, F32, 1, 3),
    (33, 2, 8, 16, F16, F32, 0, 1),
])
def test_dense_product(height, transpose, act, m, e, k, n, dtype, out_dtype, list_type, spare):
    _dense_case(m + k, m, e, k, n, dtype, out_dtype, transpose, act, list_type, spare, tuning=[0, height])


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("cap", [1, 3, 8, 17])
@pytest.mark.parametrize("height", [32, 128, 256])
def test_dense_product_on_few_workgroups(transpose, cap, height):
    """Each workgroup runs many tiles through the continuous copy stream."""
    _dense_case(cap, 700, 6, 136, 648, BF16, BF16, transpose, None, 1, 5, tuning=[0, height, cap])


@pytest.mark.parametrize("m,e,k,n", [(1, 1, 64, 64), (1, 7, 2048, 264), (2, 1024, 16, 8), (40, 70, 520, 1048),
                                     (4100, 2, 200, 304)])
@pytest.mark.parametrize("transpose", [False, True])
def test_dense_product_chosen_tiles(m, e, k, n, transpose):
    _dense_case(m, m, e, k, n, BF16, BF16, transpose, None, 0, 0, empty=0.5 if e > 1 else 0.0)


def _mx_operand(rng, shape, fmt, scale=1.0):
    v = rng.standard_normal(shape) * scale * np.exp(rng.standard_normal(shape[-1]))
    code, s = R.encode(v.astype(np.float32), fmt)
    return R.pack(code, s, fmt)


def _mx_case(seed, m, e, k, n, fmt, out_dtype, act, list_type, spare, tuning=None, empty=0.3, wide=False):
    rng = np.random.default_rng(seed)
    counts = R.counts_for(rng, m, e, empty, spare)
    gl = R.as_list(counts, list_type)
    x, xs = _mx_operand(rng, (m, k), fmt)
    w, ws = _mx_operand(rng, (e, n, k), "fp4", k ** -0.5)
    ends = np.cumsum(counts)
    xs.view(torch.uint8)[ends[-1]:] = 255  # NaN scales behind the last group
    ws.view(torch.uint8)[np.flatnonzero(counts == 0)] = 255
    xv, wv = R.decode(x, xs), R.decode(w, ws)
    want, s = R.product(xv, wv.transpose(1, 2), gl.numpy(), list_type)
    err = s * (k // 32 + 32) * R.U
    if fmt == "fp8":
        xe, xsv, we, wsv = R.elements(x), R.scale_values(xs), R.elements(w), R.scale_values(ws)
        for g, (a, b) in enumerate(R.groups(gl.numpy(), m, list_type)):
            if b > a:
                err[a:b] += R.mx_block_loss(xe[a:b], xsv[a:b], we[g], wsv[g])
    if act == "swiglu":
        want, err = R.swiglu(want, err)
    out = torch.full((m, n // 2 if act else n), SENTINEL, dtype=out_dtype, device="cuda")
    y = B.grouped_matmul(x.cuda(), w.cuda(), gl.cuda(), x_scale=xs.cuda(), w_scale=ws.cuda(), out=out, transpose_w=True,
                         activation=act, group_list_type=list_type, tuning_config=tuning)
    end = int(counts.sum())
    _check_product(y, want, err, out_dtype, end, m)
    # the bound is a worst case: a wrong scale or pairing would hide in it where it is wide
    d = (y.double().cpu() - want)[:end]
    rel = float(d.norm() / want[:end].norm()) if end else 0.0
    assert rel <= (2 ** -13 if out_dtype == F32 else 2 ** -8), rel


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("m,e,k,n,out_dtype,list_type,spare", [
    (301, 5, 576, 336, BF16, 0, 7),
    (65, 3, 64, 528, F32, 1, 0),
    (97, 9, 1088, 80, F16, 1, 3),
    (270, 2, 2048, 272, F32, 0, 1),
    (33, 4, 192, 16, BF16, 1, 2),
])
def test_mx_product(height, fmt, act, m, e, k, n, out_dtype, list_type, spare):
    _mx_case(m + k, m, e, k, n, fmt, out_dtype, act, list_type, spare, tuning=[0, height])


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("cap", [1, 3, 8])
@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("k", [64, 320, 1152])
def test_mx_product_on_few_workgroups(fmt, cap, height, k):
    _mx_case(cap + k, 500, 6, k, 400, fmt, F32, None, 1, 5, tuning=[0, height, cap])


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("m,e,k,n", [(1, 1, 64, 64), (1, 7, 2112, 264), (2, 1024, 64, 8), (1030, 3, 640, 520)])
def test_mx_product_chosen_tiles(fmt, m, e, k, n):
    _mx_case(m, m, e, k, n, fmt, BF16, None, 0, 0, empty=0.5 if e > 1 else 0.0)


@pytest.mark.parametrize("height", [128, 256])
@pytest.mark.parametrize("m,e,k,n,dtype,out_dtype,list_type,spare,empty", [
    (301, 5, 264, 336, BF16, F32, 0, 7, 0.3),
    (517, 3, 72, 528, F16, F16, 1, 0, 0.0),
    (97, 9, 520, 80, BF16, BF16, 1, 3, 0.6),
    (1, 4, 8, 16, F16, F32, 0, 0, 0.9),
    (2050, 2, 136, 144, BF16, F32, 1, 2, 0.0),
])
def test_wgrad(height, m, e, k, n, dtype, out_dtype, list_type, spare, empty):
    rng = np.random.default_rng(m + k)
    counts = R.counts_for(rng, m, e, empty, spare)
    gl = R.as_list(counts, list_type)
    x, dy = _rand(rng, (m, k), dtype), _rand(rng, (m, n), dtype, 0.1)
    _poison_outside(x, np.cumsum(counts))
    _poison_outside(dy, np.cumsum(counts))
    want, s, rows = R.wgrad(x.double(), dy.double(), gl.numpy(), list_type)
    bound = s * (rows + 1)[:, None, None] * R.U
    for cap in (0, 1, 5):
        dw = B.grouped_matmul_wgrad(x.cuda(), dy.cuda(), gl.cuda(), out_dtype=out_dtype, group_list_type=list_type,
                                    tuning_config=[0, height, cap])
        assert dw.dtype == out_dtype
        R.assert_within(dw, want, bound + R.half_step(want.abs() + bound, out_dtype), f"wgrad, cap {cap}")
        assert (dw.cpu()[counts == 0] == 0).all()
    if out_dtype == F32:
        old = _rand(rng, (e, k, n), F32)
        dw = B.grouped_matmul_wgrad(x.cuda(), dy.cuda(), gl.cuda(), out=old.cuda(), accumulate=True,
                                    group_list_type=list_type, tuning_config=[0, height])
        total = want + old.double()
        R.assert_within(dw, total, bound + R.half_step(total.abs() + bound, F32), "accumulated")
        assert torch.equal(dw.cpu()[counts == 0], old[counts == 0])


def test_wgrad_without_rows_is_zero():
    x = torch.empty((0, 64), dtype=BF16, device="cuda")
    dy = torch.empty((0, 128), dtype=BF16, device="cuda")
    gl = torch.zeros(3, dtype=torch.int64, device="cuda")
    dw = torch.full((3, 64, 128), float("nan"), dtype=F32, device="cuda")
    B.grouped_matmul_wgrad(x, dy, gl, out=dw)
    assert (dw == 0).all()


def test_wgrad_is_the_gradient_by_differences():
    """dw against central differences of sum(dy * y) in the library's own
    product.  y is linear in w, so a difference of y is exact but for y's
    rounding to fp32 and the sums' own errors (bounded as above)."""
    rng = np.random.default_rng(5)
    m, e, k, n = 90, 3, 40, 48
    gl = torch.tensor([50, 0, 40])
    x, w = _rand(rng, (m, k), BF16), _rand(rng, (e, k, n), BF16)
    dy = _rand(rng, (m, n), BF16)
    dw = B.grouped_matmul_wgrad(x.cuda(), dy.cuda(), gl.cuda(), group_list_type=1).cpu().double()
    for g, p, j in [(0, 0, 0), (0, 39, 47), (2, 17, 20), (1, 3, 3)]:
        h, total = 0.5, []
        moved = []
        for sign in (1, -1):
            v = w.clone()
            v[g, p, j] = float(w[g, p, j]) + sign * h
            moved.append(float(v[g, p, j]))
            y = B.grouped_matmul(x.cuda(), v.cuda(), gl.cuda(), out_dtype=F32, group_list_type=1,
                                 out=torch.empty((m, n), dtype=F32, device="cuda"))
            total.append((dy.double() * y.cpu().double()).sum())
        s = float((dy.double().abs() * (x.double().abs() @ w.double().abs().amax(0) + x.double().abs().sum(1, keepdim=True))).sum())
        assert abs(float(total[0] - total[1]) / (moved[0] - moved[1]) - float(dw[g, p, j])) <= 2 * s * (k + 2) * R.U / (moved[0] - moved[1]) + 1e-5


def test_row_gradient_is_the_transposed_product():
    """dx = dy w^T: the product with transpose_w, by the formula."""
    rng = np.random.default_rng(6)
    m, e, k, n = 150, 4, 136, 264
    counts = R.counts_for(rng, m, e, 0.2)
    gl = R.as_list(counts, 1)
    w, dy = _rand(rng, (e, k, n), BF16, 0.1), _rand(rng, (m, n), BF16)
    dx = B.grouped_matmul(dy.cuda(), w.cuda(), gl.cuda(), transpose_w=True, group_list_type=1)
    want, s = R.product(dy.double(), w.double().transpose(1, 2), gl.numpy(), 1)
    bound = s * (n + 1) * R.U
    R.assert_within(dx, want, bound + R.half_step(want.abs() + bound, BF16), "dx")


@pytest.mark.parametrize("list_type,gl", [(0, [40, 10, 90, 500]), (1, [30, -5, 60, 10 ** 12])])
def test_broken_group_list_stays_inside(list_type, gl):
    """Ends past m, decreasing or negative entries: read clamped, guards around y untouched."""
    rng = np.random.default_rng(8)
    m, e, k, n = 120, 4, 72, 88
    x, w = _rand(rng, (m, k), BF16), _rand(rng, (e, k, n), BF16, 0.1)
    want, s = R.product(x.double(), w.double(), np.array(gl), list_type)
    big = torch.full((m + 64, n), SENTINEL, dtype=BF16, device="cuda")
    for height in (32, 128, 256):
        big.fill_(SENTINEL)
        B.grouped_matmul(x.cuda(), w.cuda(), torch.tensor(gl).cuda(), out=big[32:32 + m], group_list_type=list_type,
                         tuning_config=[0, height])
        assert (big[:32] == SENTINEL).all() and (big[32 + m:] == SENTINEL).all()
        end = int(R.clamped_ends(gl, m, list_type)[-1])
        bound = s * (k + 1) * R.U
        R.assert_within(big[32:32 + end], want[:end], (bound + R.half_step(want.abs() + bound, BF16))[:end])


def test_infinities_and_nan_stay_in_their_rows_and_columns():
    rng = np.random.default_rng(9)
    m, e, k, n = 70, 2, 64, 72
    gl = torch.tensor([33, 37])
    x, w = _rand(rng, (m, k), BF16), _rand(rng, (e, n, k), BF16)
    x[5, 3] = float("nan")
    x[40, 0] = float("inf")
    w[1, 7, 9] = float("nan")
    y = B.grouped_matmul(x.cuda(), w.cuda(), gl.cuda(), transpose_w=True, group_list_type=1).float().cpu()
    bad = torch.zeros((m, n), dtype=torch.bool)
    bad[5] = bad[40] = True
    bad[33:, 7] = True
    assert torch.equal(~torch.isfinite(y), bad)


def test_zero_scale_codes_and_nan_scales():
    """A NaN row scale makes its row NaN where a code meets it, and no other row."""
    rng = np.random.default_rng(10)
    m, e, k, n = 40, 1, 192, 64
    x, xs = _mx_operand(rng, (m, k), "fp4")
    w, ws = _mx_operand(rng, (e, n, k), "fp4")
    xs.view(torch.uint8)[11, 2, 1] = 255
    y = B.grouped_matmul(x.cuda(), w.cuda(), torch.tensor([m]).cuda(), x_scale=xs.cuda(), w_scale=ws.cuda(),
                         transpose_w=True).float().cpu()
    assert torch.isnan(y[11]).all()
    y[11] = 0
    assert torch.isfinite(y).all()


def test_offsets_past_32_bits():
    """y of 4.3e9 elements and dw of 2.2e9: sampled rows against the formula."""
    rng = np.random.default_rng(11)
    m, e, k, n = 70000, 2, 16, 61440
    x, w = _rand(rng, (m, k), BF16), _rand(rng, (e, k, n), BF16)
    gl = torch.tensor([1000, 69000])
    y = B.grouped_matmul(x.cuda(), w.cuda(), gl.cuda(), group_list_type=1)
    for i in (0, 999, 1000, 34952, 34953, 69999):
        want = x[i].double() @ w[0 if i < 1000 else 1].double()
        s = x[i].double().abs() @ w[0 if i < 1000 else 1].double().abs()
        bound = s * (k + 1) * R.U
        R.assert_within(y[i], want, bound + R.half_step(want.abs() + bound, BF16), f"row {i}")
    del y
    x, dy = _rand(rng, (300, 36000), BF16), _rand(rng, (300, 30000), BF16)
    gl = torch.tensor([100, 200])
    dw = B.grouped_matmul_wgrad(x.cuda(), dy.cuda(), gl.cuda(), group_list_type=1, out_dtype=BF16)
    for p in (0, 17000, 35999):
        want = x[100:, p].double() @ dy[100:].double()
        s = x[100:, p].double().abs() @ dy[100:].double().abs()
        bound = s * 201 * R.U
        R.assert_within(dw[1, p], want, bound + R.half_step(want.abs() + bound, BF16), f"dw row {p}")


def test_other_stream_and_graph_replays():
    """A call on a side stream, and replays of a captured run of three calls
    with new inputs and eager work between them."""
    rng = np.random.default_rng(12)
    m, e, k, n = 260, 4, 256, 512
    gl = torch.tensor([100, 0, 60, 100]).cuda()
    x, w = _rand(rng, (m, k), BF16).cuda(), _rand(rng, (e, k, n), BF16, 0.1).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = B.grouped_matmul(x, w, gl, group_list_type=1, stream=side)
    side.synchronize()
    assert torch.equal(a, B.grouped_matmul(x, w, gl, group_list_type=1))

    def run():
        y = B.grouped_matmul(x, w, gl, group_list_type=1, activation="swiglu")
        codes, scales = B.mx_quantize(y, format="fp8")
        return y, B.mx_dequantize(codes, scales), B.grouped_matmul_wgrad(x, y, gl, group_list_type=1)
    run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = run()
    for step in range(4):
        x.copy_(_rand(rng, (m, k), BF16))
        for t in got:
            t.fill_(float("nan"))
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, v in zip(got, want):
            assert torch.equal(t, v), step


def test_results_do_not_depend_on_the_grid():
    rng = np.random.default_rng(13)
    m, e, k, n = 900, 5, 320, 400
    gl = R.as_list(R.counts_for(rng, m, e), 1).cuda()
    x, w = _rand(rng, (m, k), BF16).cuda(), _rand(rng, (e, k, n), BF16).cuda()
    for height in (32, 128, 256):
        first = B.grouped_matmul(x, w, gl, group_list_type=1, tuning_config=[0, height])
        for cap in (1, 7, 64):
            assert torch.equal(first, B.grouped_matmul(x, w, gl, group_list_type=1, tuning_config=[0, height, cap]))


@pytest.mark.parametrize("height", [32, 128, 256])
def test_groups_without_any_row(height):
    """m > 0 and every group empty: nothing is written; the weight gradient is zero."""
    x = torch.ones((50, 64), dtype=BF16, device="cuda")
    w = torch.ones((3, 64, 32), dtype=BF16, device="cuda")
    gl = torch.zeros(3, dtype=torch.int64, device="cuda")
    out = torch.full((50, 32), SENTINEL, dtype=BF16, device="cuda")
    for list_type in (0, 1):
        B.grouped_matmul(x, w, gl, out=out, group_list_type=list_type, tuning_config=[0, height])
        assert (out == SENTINEL).all()
        if height > 32:
            dw = B.grouped_matmul_wgrad(x, x[:, :32].contiguous(), gl, group_list_type=list_type, tuning_config=[0, height])
            assert (dw == 0).all()


@pytest.mark.parametrize("height", [32, 128, 256])
def test_as_many_experts_as_allowed(height):
    _dense_case(21, 3000, 1024, 72, 40, BF16, BF16, False, None, 1, 2, tuning=[0, height], empty=0.4)
    for fmt in ("fp4", "fp8"):
        _mx_case(22, 3000, 1024, 128, 48, fmt, BF16, None, 0, 2, tuning=[0, height], empty=0.4)


def test_weight_gradient_of_as_many_experts_as_allowed():
    rng = np.random.default_rng(23)
    m, e, k, n = 3000, 1024, 24, 40
    counts = R.counts_for(rng, m, e, 0.4)
    x, dy = _rand(rng, (m, k), BF16), _rand(rng, (m, n), BF16)
    want, s, rows = R.wgrad(x.double(), dy.double(), counts, 1)
    bound = s * (rows + 1)[:, None, None] * R.U
    for height in (128, 256):
        dw = B.grouped_matmul_wgrad(x.cuda(), dy.cuda(), torch.from_numpy(counts).cuda(), group_list_type=1,
                                    tuning_config=[0, height])
        R.assert_within(dw, want, bound + R.half_step(want.abs() + bound, F32), f"height {height}")


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("height", [32, 128, 256])
def test_nan_scales_stay_in_their_row_or_column(fmt, height):
    rng = np.random.default_rng(24)
    m, e, k, n = 300, 2, 1088, 272
    x, xs = _mx_operand(rng, (m, k), fmt)
    w, ws = _mx_operand(rng, (e, n, k), "fp4")
    xs.view(torch.uint8)[11, 16, 0] = 255
    xs.view(torch.uint8)[12, 0, 0] = 255
    ws.view(torch.uint8)[1, 5, 16, 1] = 255
    y = B.grouped_matmul(x.cuda(), w.cuda(), torch.tensor([100, 200]).cuda(), x_scale=xs.cuda(), w_scale=ws.cuda(),
                         transpose_w=True, group_list_type=1, tuning_config=[0, height]).float().cpu()
    bad = torch.zeros((m, n), dtype=torch.bool)
    bad[11] = bad[12] = True
    bad[100:, 5] = True
    assert torch.equal(torch.isnan(y), bad)


@pytest.mark.parametrize("seed", range(40))
def test_drawn_products(seed):
    """Shapes, layouts, types, tiles and group lists drawn over small ranges."""
    rng = np.random.default_rng(1000 + seed)
    m, e = int(rng.integers(1, 900)), int(rng.integers(1, 40))
    height, cap = int(rng.choice([0, 32, 128, 256])), int(rng.choice([0, 0, 5, 40]))
    spare = int(rng.integers(0, min(m, 9)))
    act = [None, "swiglu"][rng.integers(2)]
    list_type = int(rng.integers(2))
    if rng.random() < 0.5:
        k, n = 8 * int(rng.integers(1, 90)), 16 * int(rng.integers(1, 50))
        dtype = [BF16, F16][rng.integers(2)]
        _dense_case(seed, m, e, k, n, dtype, [dtype, F32][rng.integers(2)], bool(rng.integers(2)), act, list_type, spare,
                    tuning=[0, height, cap])
    else:
        k, n = 64 * int(rng.integers(1, 30)), 16 * int(rng.integers(1, 50))
        _mx_case(seed, m, e, k, n, ["fp4", "fp8"][rng.integers(2)], [BF16, F16, F32][rng.integers(3)], act, list_type,
                 spare, tuning=[0, height, cap])
