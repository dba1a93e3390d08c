"""The gated feed-forward block, forward and back, against plain 64-bit forms,
within bounds derived in gated_ref.py and grouped_ref.py."""
import numpy as np
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import gated_ref as G
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
SENTINEL = 7.25


def _rand(rng, shape, dtype, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(dtype)


def _quantised(x):
    return R.pack(*R.encode(x.float().numpy(), "fp8"), "fp8")


def _bytes(t):
    return t.cpu().view(torch.uint8)


def _within(got, want, bound, end, what):
    dtype = got.dtype
    R.assert_within(got.cpu()[:end], want[:end], (bound + R.half_step(want.abs() + bound, dtype))[:end], what)
    assert (got.cpu()[end:] == SENTINEL).all(), f"{what}: rows behind the last group were written"


def _outputs(m, f, dtype, keep):
    """Buffers full of a sentinel."""
    kept = scale = None
    if keep == "full":
        kept = torch.full((m, 2 * f), SENTINEL, dtype=dtype, device="cuda")
    elif keep == "fp8":
        kept = torch.full((m, 2 * f), 0x5A, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        scale = torch.full((m, 2 * f // 64, 2), 0x5A, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    return torch.full((m, f), SENTINEL, dtype=dtype, device="cuda"), kept, scale


def _forward_case(seed, m, e, k, f, dtype, transpose, act, keep, list_type, spare, tuning=None, empty=0.3):
    rng = np.random.default_rng(seed)
    counts = R.counts_for(rng, m, e, empty, spare)
    end = int(counts.sum())
    gl = R.as_list(counts, list_type)
    x = _rand(rng, (m, k), dtype)
    w = _rand(rng, (e, 2 * f, k) if transpose else (e, k, 2 * f), dtype, 1.5 * k ** -0.5)
    x[end:] = float("nan")
    w[counts == 0] = float("inf")  # an expert without rows is never read
    both, s = R.product(x.double(), (w.transpose(1, 2) if transpose else w).double(), gl.numpy(), list_type)
    err = s * (k + 1) * R.U
    want, bound = G.forward(both, err, act)
    out, kept, scale = _outputs(m, f, dtype, keep)
    h, kept, scale = B.gated_matmul(x.cuda(), w.cuda(), gl.cuda(), activation=act, keep=keep, out=out, kept=kept,
                                    kept_scale=scale, transpose_w=transpose, group_list_type=list_type, tuning_config=tuning)
    assert h is out
    _within(h, want, bound, end, "h")
    if keep == "full":
        _within(kept, both, err, end, "kept")
    elif keep == "fp8":
        v = R.decode(kept.cpu(), scale.cpu())
        R.assert_within(v[:end], both[:end], G.fp8_bound(both[:end], err[:end]), "kept")
        assert (_bytes(kept)[end:] == 0x5A).all() and (_bytes(scale)[end:] == 0x5A).all()
    else:
        assert kept is None and scale is None


def _backward_case(seed, m, e, d, f, dtype, transpose, act, keep, list_type, spare, tuning=None, empty=0.3, want_h=True):
    rng = np.random.default_rng(seed)
    counts = R.counts_for(rng, m, e, empty, spare)
    end = int(counts.sum())
    gl = R.as_list(counts, list_type)
    dy = _rand(rng, (m, d), dtype, 0.1)
    w = _rand(rng, (e, f, d) if transpose else (e, d, f), dtype, d ** -0.5)
    both = _rand(rng, (m, 2 * f), dtype, 2.0)
    dy[end:] = float("nan")
    w[counts == 0] = float("nan")
    kept, scale = (both.clone(), None) if keep == "full" else _quantised(both)
    if keep == "full":
        kept[end:] = float("inf")
    else:
        scale.view(torch.uint8)[end:] = 255
    values = both.double() if keep == "full" else R.decode(kept, scale)
    dh, s = R.product(dy.double(), (w.transpose(1, 2) if transpose else w).double(), gl.numpy(), list_type)
    want, bound, h_want, h_bound = G.backward(dh, s * (d + 1) * R.U, values, act)
    out = torch.full((m, 2 * f), SENTINEL, dtype=dtype, device="cuda")
    h = torch.full((m, f), SENTINEL, dtype=dtype, device="cuda") if want_h else None
    got, got_h = B.gated_matmul_backward(dy.cuda(), w.cuda(), gl.cuda(), kept.cuda(), kept_scale=None if scale is None else scale.cuda(),
                                         activation=act, out=out, h=h, want_h=want_h, transpose_w=transpose,
                                         group_list_type=list_type, tuning_config=tuning)
    assert got is out and got_h is h
    _within(got, want, bound, end, "gradients")
    if want_h:
        _within(h, h_want, h_bound, end, "h again")


SHAPES = [  # m, e, k or d, f, dtype, list type, spare rows
    (301, 5, 264, 160, BF16, 0, 7),
    (517, 3, 72, 288, F16, 1, 0),
    (97, 9, 1032, 32, BF16, 1, 3),
    (33, 2, 8, 64, F16, 0, 1),
    (1, 1, 64, 96, BF16, 1, 0),
]


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("keep", [None, "full", "fp8"])
def test_forward(height, transpose, act, keep):
    for i, (m, e, k, f, dtype, list_type, spare) in enumerate(SHAPES):
        _forward_case(i, m, e, k, f, dtype, transpose, act, keep, list_type, spare, tuning=[0, height])


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("keep", ["full", "fp8"])
def test_backward(height, transpose, act, keep):
    for i, (m, e, d, f, dtype, list_type, spare) in enumerate(SHAPES):
        _backward_case(50 + i, m, e, d, f, dtype, transpose, act, keep, list_type, spare, tuning=[0, height],
                       want_h=i != 2)


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("f", [8, 24, 40, 136, 264])
def test_columns_that_end_inside_a_block(height, f):
    """f a multiple of 8 only: nothing kept, or in 16 bits."""
    for transpose in (False, True):
        for keep in (None, "full"):
            _forward_case(f, 210, 3, 136, f, BF16, transpose, "swiglu", keep, 1, 2, tuning=[0, height])
        _backward_case(f, 210, 3, 136, f, F16, transpose, "geglu", "full", 0, 2, tuning=[0, height])


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("cap", [1, 3, 16])
def test_on_few_workgroups(height, cap):
    """Every workgroup has many tiles, so that copies, sums and what was kept
    of one tile run into the next."""
    _forward_case(3, 700, 6, 200, 416, BF16, False, "swiglu", "fp8", 1, 5, tuning=[0, height, cap])
    _backward_case(4, 700, 6, 200, 416, BF16, True, "swiglu", "fp8", 1, 5, tuning=[0, height, cap])
    _backward_case(5, 700, 6, 200, 416, F16, False, "geglu", "full", 0, 5, tuning=[0, height, cap])


def _exact_sums(rng, m, e, k, f):
    """Operands of small whole numbers, and per column a power of two: every sum
    is exact in fp32 whatever its order."""
    x = torch.from_numpy(rng.integers(-4, 5, (m, k))).to(BF16)
    w = torch.from_numpy(rng.integers(-3, 4, (e, k, 2 * f)) * 2.0 ** rng.integers(-6, 7, (e, 1, 2 * f))).to(BF16)
    return x, w


@pytest.mark.parametrize("height", [32, 128, 256])
def test_what_is_kept_in_fp8_is_what_mx_quantisation_gives(height):
    """Codes and scales to the bit, where the sums are exact: rows of zeros and
    saturated values (448 to 512 of the scale) among them."""
    rng = np.random.default_rng(8)
    m, e, k, f = 150, 3, 64, 224
    x, w = _exact_sums(rng, m, e, k, f)
    x[7] = 0
    counts = np.array([70, 0, 80])
    both, _ = R.product(x.double(), w.double(), counts, 1)
    codes, scales = R.pack(*R.encode(both.float().numpy(), "fp8"), "fp8")
    _, kept, scale = B.gated_matmul(x.cuda(), w.cuda(), torch.from_numpy(counts).cuda(), keep="fp8", group_list_type=1,
                                    tuning_config=[0, height])
    assert torch.equal(_bytes(scale), _bytes(scales))
    # (a code's sign is the sum's; a sum of zero has none to speak of)
    zero = (_bytes(kept) & 127) == 0
    assert torch.equal(zero, (_bytes(codes) & 127) == 0)
    assert torch.equal(_bytes(kept)[~zero], _bytes(codes)[~zero])
    # and it is what the library's own quantisation makes of them
    c, s = B.mx_quantize(both.float().cuda(), format="fp8")
    assert torch.equal(_bytes(s), _bytes(scale)) and torch.equal(_bytes(c)[~zero], _bytes(kept)[~zero])


def test_swiglu_is_grouped_matmuls():
    """The same sums, the same gate: to the bit, kept or not."""
    rng = np.random.default_rng(9)
    m, e, k, f = 400, 4, 328, 192
    x, w = _rand(rng, (m, k), BF16).cuda(), _rand(rng, (e, k, 2 * f), BF16, 0.2).cuda()
    gl = torch.tensor([100, 0, 200, 100]).cuda()
    for height in (32, 128, 256):
        t = [0, height]
        want = B.grouped_matmul(x, w, gl, activation="swiglu", group_list_type=1, tuning_config=t)
        for keep in (None, "full", "fp8"):
            assert torch.equal(B.gated_matmul(x, w, gl, keep=keep, group_list_type=1, tuning_config=t)[0], want)


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("height", [32, 128, 256])
def test_gates_of_every_size(act, height):
    """Gates from -1e30 to 1e30 and through the range where exp(-z) passes
    fp32's, beside ups and gradients small and large."""
    sizes = torch.tensor([0.0, 1e-30, 1e-6, 0.3, 1.0, 1.2785, 3.0, 5.5, 9.0, 9.98, 10.0, 10.2, 11.0, 12.5, 15.9, 16.1, 30.0, 60.0,
                          80.0, 86.0, 87.0, 87.25, 87.5, 88.0, 88.75, 90.0, 100.0, 120.0, 170.0, 1e3, 1e10, 1e30])
    g = torch.cat((sizes, -sizes)).to(BF16)
    up = torch.tensor([1.0, -2.0 ** 20, 2.0 ** -20, 2.0 ** 100]).to(BF16)
    m, f = len(up), len(g)
    both = torch.cat((g.expand(m, f), up[:, None].expand(m, f)), 1).contiguous()
    # forward: one row of x picks one row of w
    x, w = torch.eye(m, dtype=BF16), both[None]
    gl = torch.tensor([m])
    x8, w8 = torch.zeros((m, 8), dtype=BF16), torch.zeros((1, 8, 2 * f), dtype=BF16)
    x8[:, :m], w8[:, :m] = x, w
    # fp32 flushes what is below 2^-126, and keeps few bits just above it
    floor = 2.0 ** -126
    want, bound = G.forward(both.double(), torch.zeros(m, 2 * f, dtype=torch.float64), act)
    want32 = want.clamp(-3.4e38, 3.4e38)
    h, _, _ = B.gated_matmul(x8.cuda(), w8.cuda(), gl.cuda(), activation=act, tuning_config=[0, height])
    fine = want.abs() < 3e38
    R.assert_within(torch.where(fine, h.cpu().double(), want32), want32, bound + R.half_step(want.abs(), BF16) + floor, "h")
    # back: dh is dy where the weights are one
    for dh in (1.0, 2.0 ** -30, -2.0 ** 15):
        dy = torch.zeros((m, 8), dtype=BF16)
        dy[:, 0] = dh
        ones = torch.ones((1, f, 8), dtype=BF16)
        want, bound, h_want, h_bound = G.backward(torch.full((m, f), dh, dtype=torch.float64), torch.zeros(m, f, dtype=torch.float64),
                                                  both.double(), act)
        d, h = B.gated_matmul_backward(dy.cuda(), ones.cuda(), gl.cuda(), both.cuda(), activation=act, tuning_config=[0, height])
        for got, ref, b in ((d, want, bound), (h, h_want, h_bound)):
            # products of three may pass fp32's range on the way: 2^100 2^15 1e30
            fine = ref.abs() < 3e38
            R.assert_within(torch.where(fine, got.cpu().double(), ref), ref, b + R.half_step(ref.abs(), BF16) + floor, "back")


@pytest.mark.parametrize("height", [32, 128, 256])
def test_infinities_and_nan_stay_in_their_places(height):
    m, e, k, f = 90, 2, 64, 64
    rng = np.random.default_rng(12)
    x, w = _rand(rng, (m, k), BF16), _rand(rng, (e, k, 2 * f), BF16, 0.2)
    x[5] = float("nan")
    w[1, :, 3] = float("inf")        # a gate column of the second expert: +-inf or NaN
    w[1, :, f + 40] = float("nan")   # an up column
    gl = torch.tensor([50, 40]).cuda()
    h, kept, scale = B.gated_matmul(x.cuda(), w.cuda(), gl, keep="fp8", group_list_type=1, tuning_config=[0, height])
    h = h.float().cpu()
    bad = torch.zeros((m, f), dtype=torch.bool)
    bad[5] = True
    bad[50:, 40] = True
    assert torch.isnan(h[bad]).all()
    bad[50:, 3] = True
    assert torch.isfinite(h[~bad]).all()
    # whole blocks of what is kept become NaN: row 5; columns 0..31 and f+32..f+63 of the second expert
    v = B.mx_dequantize(kept, scale).float().cpu()
    lost = torch.zeros((m, 2 * f), dtype=torch.bool)
    lost[5] = True
    lost[50:, :32] = True
    lost[50:, f + 32:] = True
    assert torch.equal(torch.isnan(v), lost)
    assert ((_bytes(kept)[lost]) == 0).all()
    # back: NaN where a kept value is, or where dy is
    dy, wd = _rand(rng, (m, 32), BF16), _rand(rng, (e, f, 32), BF16)
    dy[7] = float("nan")
    d, hb = B.gated_matmul_backward(dy.cuda(), wd.cuda(), gl, kept, kept_scale=scale, group_list_type=1, tuning_config=[0, height])
    gate_bad, up_bad = lost[:, :f], lost[:, f:]
    assert torch.equal(torch.isnan(hb.float().cpu()), gate_bad | up_bad)
    both = gate_bad | up_bad
    both[7] = True
    alone = gate_bad.clone()
    alone[7] = True
    assert torch.equal(torch.isnan(d.float().cpu()), torch.cat((both, alone), 1))


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("keep", ["full", "fp8"])
def test_gradients_by_differences(act, keep):
    """The gradients of u and v against central differences of sum(dy (h w)) in
    64 bits: the step's own error is its third derivative's, below 6 step^2."""
    rng = np.random.default_rng(14)
    m, e, d, f = 40, 2, 48, 64
    counts = np.array([25, 15])
    dy, w = _rand(rng, (m, d), BF16), _rand(rng, (e, f, d), BF16, d ** -0.5)
    both = _rand(rng, (m, 2 * f), BF16, 1.5)
    kept, scale = (both, None) if keep == "full" else _quantised(both)
    values = both.double() if keep == "full" else R.decode(kept, scale)
    got, _ = B.gated_matmul_backward(dy.cuda(), w.cuda(), torch.from_numpy(counts).cuda(), kept.cuda(),
                                     kept_scale=None if scale is None else scale.cuda(), activation=act, group_list_type=1)
    dh, s = R.product(dy.double(), w.double().transpose(1, 2), counts, 1)
    zero = torch.zeros_like(values)
    step = 1e-4

    def value(at):  # what each (u, v) adds to the loss
        return dh * G.forward(at, zero, act)[0]
    diff = torch.empty_like(values)
    for half in (0, 1):
        move = torch.zeros_like(values)
        move[:, half * f:(half + 1) * f] = step
        diff[:, half * f:(half + 1) * f] = (value(values + move) - value(values - move)) / (2 * step)
    _, bound, _, _ = G.backward(dh, s * (d + 1) * R.U, values, act)
    bound = bound + 6 * step ** 2 * torch.cat((dh * values[:, f:], dh * values[:, :f]), 1).abs() + 1e-9 * (1 + dh.abs().repeat(1, 2))
    R.assert_within(got, diff, bound + R.half_step(diff.abs() + bound, BF16), "differences")


@pytest.mark.parametrize("list_type,gl", [(0, [50, 30, 90]), (0, [-5, 40, 500]), (1, [30, -9, 60]), (1, [60, 60, 60]), (0, [0, 0, 0]), (1, [0, 0, 0])])
@pytest.mark.parametrize("height", [32, 128, 256])
def test_broken_group_lists_stay_inside(list_type, gl, height):
    rng = np.random.default_rng(15)
    m, e, k, f = 100, 3, 72, 64
    ends = R.clamped_ends(gl, m, list_type)
    x, w = _rand(rng, (m, k), BF16), _rand(rng, (e, k, 2 * f), BF16, 0.2)
    both, s = R.product(x.double(), w.double(), gl, list_type)
    want, bound = G.forward(both, s * (k + 1) * R.U, "swiglu")
    out, kept, scale = _outputs(m, f, BF16, "full")
    g = torch.tensor(gl).cuda()
    B.gated_matmul(x.cuda(), w.cuda(), g, keep="full", out=out, kept=kept, group_list_type=list_type, tuning_config=[0, height])
    _within(out, want, bound, int(ends[-1]), "h")
    _within(kept, both, s * (k + 1) * R.U, int(ends[-1]), "kept")
    wd = _rand(rng, (e, f, k), BF16, 0.2)
    dh, s = R.product(x.double(), wd.double().transpose(1, 2), gl, list_type)
    values = _rand(rng, (m, 2 * f), BF16)
    want, bound, h_want, h_bound = G.backward(dh, s * (k + 1) * R.U, values.double(), "swiglu")
    d = torch.full((m, 2 * f), SENTINEL, dtype=BF16, device="cuda")
    out.fill_(SENTINEL)
    B.gated_matmul_backward(x.cuda(), wd.cuda(), g, values.cuda(), out=d, h=out, group_list_type=list_type, tuning_config=[0, height])
    _within(d, want, bound, int(ends[-1]), "gradients")
    _within(out, h_want, h_bound, int(ends[-1]), "h again")


@pytest.mark.parametrize("seed", range(48))
def test_drawn(seed):
    rng = np.random.default_rng(3000 + seed)
    m, e = int(rng.integers(1, 900)), int(rng.integers(1, 40))
    height, cap = int(rng.choice([0, 32, 128, 256])), int(rng.choice([0, 0, 5, 40]))
    keep = [None, "full", "fp8"][rng.integers(3)]
    k, f = 8 * int(rng.integers(1, 90)), (32 if keep == "fp8" else 8) * int(rng.integers(1, 20))
    args = (m, e, k, f, [BF16, F16][rng.integers(2)], bool(rng.integers(2)), ["swiglu", "geglu"][rng.integers(2)])
    rest = dict(list_type=int(rng.integers(2)), spare=int(rng.integers(0, min(m, 9))), tuning=[int(rng.choice([0, 20])), height, cap])
    if keep is None or rng.random() < 0.5:
        _forward_case(seed, *args, keep, **rest)
    else:
        _backward_case(seed, *args, keep, **rest)


def test_no_rows():
    gl = torch.tensor([0, 0]).cuda()
    x, w = torch.empty((0, 64), dtype=BF16, device="cuda"), torch.ones((2, 64, 128), dtype=BF16, device="cuda")
    h, kept, scale = B.gated_matmul(x, w, gl, keep="fp8")
    assert h.shape == (0, 64) and kept.shape == (0, 128) and scale.shape == (0, 2, 2)
    d, h = B.gated_matmul_backward(x, torch.ones((2, 64, 64), dtype=BF16, device="cuda"), gl, kept, kept_scale=scale)
    assert d.shape == (0, 128) and h.shape == (0, 64)


@pytest.mark.parametrize("height", [32, 128, 256])
def test_as_many_experts_as_allowed(height):
    _forward_case(21, 3000, 1024, 72, 32, BF16, False, "swiglu", "fp8", 1, 2, tuning=[0, height], empty=0.4)
    _backward_case(22, 3000, 1024, 72, 32, BF16, True, "geglu", "fp8", 0, 2, tuning=[0, height], empty=0.4)
