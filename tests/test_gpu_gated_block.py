"""The gated block as a training step uses it: its forward pass, its way back and
the weight gradients together, inside a torch.autograd.Function, in captured
graphs, on other streams and at the largest sizes."""
import ctypes

import numpy as np
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import gated_ref as G
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def _rand(rng, shape, dtype=BF16, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(dtype)


def _check(got, want, bound, what):
    R.assert_within(got, want, bound + R.half_step(want.abs() + bound, got.dtype), what)


class Block(torch.autograd.Function):
    """y = (act(x w1[..., :f]) * (x w1[..., f:])) w2 for rows grouped by expert;
    the rows are kept in FP8 for w1's gradient, the projections as `keep` says."""

    @staticmethod
    def forward(ctx, x, w1, w2, gl, act, keep):
        h, kept, scale = B.gated_matmul(x, w1, gl, activation=act, keep=keep, group_list_type=1)
        codes, x_scale = B.mx_quantize(x, format="fp8")
        ctx.save_for_backward(codes, x_scale, kept, scale, w1, w2, gl)
        ctx.act = act
        return B.grouped_matmul(h, w2, gl, group_list_type=1)

    @staticmethod
    def backward(ctx, dy):
        codes, x_scale, kept, scale, w1, w2, gl = ctx.saved_tensors
        d, h = B.gated_matmul_backward(dy.contiguous(), w2, gl, kept, kept_scale=scale, activation=ctx.act, group_list_type=1)
        dx = B.grouped_matmul(d, w1, gl, transpose_w=True, group_list_type=1)
        dw1 = B.grouped_matmul_wgrad(codes, d, gl, x_scale=x_scale, out_dtype=BF16, group_list_type=1)
        dw2 = B.grouped_matmul_wgrad(h, dy, gl, out_dtype=BF16, group_list_type=1)
        return dx, dw1, dw2, None, None, None


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("keep", ["full", "fp8"])
@pytest.mark.parametrize("counts", [[150, 0, 93, 60], [303]])
def test_training_step(act, keep, counts):
    """Every gradient against the 64-bit form of what the stage before it gave
    (the values kept are those that the calls return)."""
    rng = np.random.default_rng(len(counts))
    m, e, k, f = 303, len(counts), 192, 160
    gl = torch.tensor(counts)
    x, w1, w2 = _rand(rng, (m, k)), _rand(rng, (e, k, 2 * f), scale=1.5 * k ** -0.5), _rand(rng, (e, f, k), scale=f ** -0.5)
    dy = _rand(rng, (m, k), scale=0.1)
    xg, w1g, w2g = (t.cuda().requires_grad_() for t in (x, w1, w2))
    y = Block.apply(xg, w1g, w2g, gl.cuda(), act, keep)
    y.backward(dy.cuda())

    # the stages again, from outside
    c = gl.cuda()
    h, kept, scale = B.gated_matmul(x.cuda(), w1.cuda(), c, activation=act, keep=keep, group_list_type=1)
    codes, x_scale = B.mx_quantize(x.cuda(), format="fp8")
    d, hb = B.gated_matmul_backward(dy.cuda(), w2.cuda(), c, kept, kept_scale=scale, activation=act, group_list_type=1)
    both, s = R.product(x.double(), w1.double(), counts, 1)
    want, bound = G.forward(both, s * (k + 1) * R.U, act)
    _check(h, want, bound, "h")
    want, s = R.product(h.cpu().double(), w2.double(), counts, 1)
    _check(y.detach(), want, s * (f + 1) * R.U, "y")
    values = kept.cpu().double() if keep == "full" else R.decode(kept.cpu(), scale.cpu())
    dh, s = R.product(dy.double(), w2.double().transpose(1, 2), counts, 1)
    want, bound, h_want, h_bound = G.backward(dh, s * (k + 1) * R.U, values, act)
    _check(d, want, bound, "gradients of the projections")
    _check(hb, h_want, h_bound, "h again")
    want, s = R.product(d.cpu().double(), w1.double().transpose(1, 2), counts, 1)
    _check(xg.grad, want, s * (2 * f + 1) * R.U, "dx")
    for got, a, b in ((w1g.grad, R.decode(codes.cpu(), x_scale.cpu()), d), (w2g.grad, hb.cpu().double(), dy)):
        want, s, rows = R.wgrad(a, b.cpu().double(), counts, 1)
        _check(got, want, s * (rows + 1)[:, None, None] * R.U, "dw")


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
def test_the_block_against_differentiation_in_64_bits(act):
    """All of it against torch's own derivative of the plain block in 64 bits.
    Kept in bf16, what the gradients are made of is off by 2^-8 of itself once
    (u, v, h) and d by another 2^-8, so that the whole stays within 2^-5 of each
    gradient's norm: u and v enter through at most three factors whose slopes are
    bounded by 1.13 and 1, rounded to 2^-8 each, with the roundings of d, h, dy's
    own and the result's, 8 half steps of 2^-8 in all."""
    rng = np.random.default_rng(21)
    m, e, k, f = 256, 2, 128, 96
    counts = [100, 156]
    x, w1, w2 = _rand(rng, (m, k)), _rand(rng, (e, k, 2 * f), scale=k ** -0.5), _rand(rng, (e, f, k), scale=f ** -0.5)
    dy = _rand(rng, (m, k))
    leaves = [t.double().requires_grad_() for t in (x, w1, w2)]
    parts = []
    for g, part in enumerate(leaves[0].split(counts)):
        u, v = (part @ leaves[1][g]).chunk(2, -1)
        a = torch.nn.functional.silu(u) if act == "swiglu" else torch.nn.functional.gelu(u, approximate="tanh")
        parts.append((a * v) @ leaves[2][g])
    torch.cat(parts).backward(dy.double())
    c = torch.tensor(counts).cuda()
    _, kept, _ = B.gated_matmul(x.cuda(), w1.cuda(), c, activation=act, keep="full", group_list_type=1)
    d, h = B.gated_matmul_backward(dy.cuda(), w2.cuda(), c, kept, activation=act, group_list_type=1)
    got = [B.grouped_matmul(d, w1.cuda(), c, transpose_w=True, group_list_type=1),
           B.grouped_matmul_wgrad(x.cuda(), d, c, group_list_type=1), B.grouped_matmul_wgrad(h, dy.cuda(), c, group_list_type=1)]
    for leaf, g in zip(leaves, got):
        assert float((g.cpu().double() - leaf.grad).norm()) <= 2.0 ** -5 * float(leaf.grad.norm())


@pytest.mark.parametrize("height", [32, 128, 256])
def test_results_do_not_depend_on_the_grid(height):
    rng = np.random.default_rng(13)
    m, e, k, f = 900, 5, 320, 224
    gl = R.as_list(R.counts_for(rng, m, e), 1).cuda()
    x, w1, w2 = _rand(rng, (m, k)).cuda(), _rand(rng, (e, k, 2 * f), scale=0.1).cuda(), _rand(rng, (e, f, k), scale=0.1).cuda()

    def run(cap):
        kw = dict(group_list_type=1, tuning_config=[0, height, cap])
        h, kept, scale = (torch.zeros((m, f), dtype=BF16, device="cuda"),
                          torch.zeros((m, 2 * f), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                          torch.zeros((m, f // 32, 2), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu))
        B.gated_matmul(x, w1, gl, keep="fp8", out=h, kept=kept, kept_scale=scale, **kw)
        d, hb = torch.zeros((m, 2 * f), dtype=BF16, device="cuda"), torch.zeros((m, f), dtype=BF16, device="cuda")
        B.gated_matmul_backward(x, w2, gl, kept, kept_scale=scale, out=d, h=hb, **kw)
        dw = []
        if height > 32:
            dw = [B.grouped_matmul_wgrad(kept, x, gl, x_scale=scale, **kw), B.grouped_matmul_wgrad(x, kept, gl, dy_scale=scale, **kw)]
        return [h, kept.view(torch.uint8), scale.view(torch.uint8), d, hb, *dw]
    first = run(0)
    for cap in (1, 7, 64):
        for a, b in zip(first, run(cap)):
            assert torch.equal(a, b)


def test_tiles_agree():
    """128-row and 256-row tiles add in one order, whatever rows are expected."""
    rng = np.random.default_rng(14)
    m, e, k, f = 700, 4, 264, 96
    gl = R.as_list(R.counts_for(rng, m, e, 0.2), 1).cuda()
    x, w1, w2 = _rand(rng, (m, k)).cuda(), _rand(rng, (e, k, 2 * f), scale=0.1).cuda(), _rand(rng, (e, f, k), scale=0.1).cuda()
    got = []
    for tuning in ([0, 128], [0, 256], [40, 128, 8], [700, 256]):
        kw = dict(group_list_type=1, tuning_config=tuning)
        h, kept, _ = B.gated_matmul(x, w1, gl, keep="full", **kw)
        got.append([h, kept, *B.gated_matmul_backward(x, w2, gl, kept, **kw)])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("m,e,k,f", [(48, 1, 512, 1024), (269, 3, 392, 256), (200, 2, 136, 800), (512, 4, 128, 2048), (512, 4, 128, 2080), (130, 3, 64, 72)])
@pytest.mark.parametrize("transpose", [False, True])
def test_chosen_tiles(m, e, k, f, transpose):
    """Few rows of small weights under the tile that the plan takes, on either
    side of its bound: results of some tile's, forward and back."""
    rng = np.random.default_rng(f + m)
    counts = R.counts_for(rng, m, e, 0.2)
    gl = torch.from_numpy(counts).cuda()
    x = _rand(rng, (m, k))
    w1 = _rand(rng, (e, 2 * f, k) if transpose else (e, k, 2 * f), scale=1.5 * k ** -0.5)
    w2 = _rand(rng, (e, f, k) if transpose else (e, k, f), scale=k ** -0.5)
    kw = dict(transpose_w=transpose, group_list_type=1)
    h, kept, _ = B.gated_matmul(x.cuda(), w1.cuda(), gl, keep="full", **kw)
    d, hb = B.gated_matmul_backward(x.cuda(), w2.cuda(), gl, kept, **kw)
    fits = []
    for height in (32, 128):
        other, also, _ = B.gated_matmul(x.cuda(), w1.cuda(), gl, keep="full", tuning_config=[0, height], **kw)
        fits.append(torch.equal(h, other) and torch.equal(kept, also))
    assert any(fits)
    both, s = R.product(x.double(), (w1.transpose(1, 2) if transpose else w1).double(), counts, 1)
    want, bound = G.forward(both, s * (k + 1) * R.U, "swiglu")
    _check(h, want, bound, "h")
    dh, s = R.product(x.double(), (w2.transpose(1, 2) if transpose else w2).double(), counts, 1)
    want, bound, h_want, h_bound = G.backward(dh, s * (k + 1) * R.U, kept.cpu().double(), "swiglu")
    _check(d, want, bound, "gradients")
    _check(hb, h_want, h_bound, "h again")


@pytest.mark.parametrize("m,e,k,f,tiles", [(20, 3, 200, 328, "thin"), (40, 5, 136, 1000, "thin"), (1, 1, 2048, 4096, "thin"),
                                           (9, 2, 72, 8, "thin"), (33, 16, 64, 640, "thin"), (40, 24, 136, 1000, "narrow"),
                                           (33, 16, 64, 1600, "narrow")])
@pytest.mark.parametrize("act", ["swiglu", "geglu"])
def test_narrow_tiles_of_both_widths(m, e, k, f, tiles, act):
    """Weights (e,n,k) under few tiles (32 columns each, a gate's and its up's in
    one block) and under more (64)."""
    rng = np.random.default_rng(f)
    counts = R.counts_for(rng, m, e, 0.2)
    gl = torch.from_numpy(counts).cuda()
    x, w1, w2 = _rand(rng, (m, k)), _rand(rng, (e, 2 * f, k), scale=1.5 * k ** -0.5), _rand(rng, (e, f, k), scale=k ** -0.5)
    kw = dict(activation=act, transpose_w=True, group_list_type=1, tuning_config=[0, 32])
    info = B.GmPlanInfo()
    dh = torch.empty((m, f), dtype=BF16, device="cuda")
    args, keepalive = B.make_gm_args(x.cuda(), w2.cuda(), gl, dh, transpose_w=True, group_list_type=1, tuning_config=[0, 32])
    assert B.lib().gmm_grouped_matmul_plan(ctypes.byref(args), ctypes.byref(info)) == B.OK
    assert info.tile_n == (32 if tiles == "thin" else 64)
    both, s = R.product(x.double(), w1.double().transpose(1, 2), counts, 1)
    want, bound = G.forward(both, s * (k + 1) * R.U, act)
    h, kept, _ = B.gated_matmul(x.cuda(), w1.cuda(), gl, keep="full", **kw)
    _check(h, want, bound, "h")
    _check(kept, both, s * (k + 1) * R.U, "kept")
    assert torch.equal(B.gated_matmul(x.cuda(), w1.cuda(), gl, **kw)[0], h)
    if f % 32 == 0:  # kept in FP8 the tiles are wider; the sums are the same
        assert torch.equal(B.gated_matmul(x.cuda(), w1.cuda(), gl, keep="fp8", **kw)[0], h)
    dh, s = R.product(x.double(), w2.double().transpose(1, 2), counts, 1)
    want, bound, h_want, h_bound = G.backward(dh, s * (k + 1) * R.U, kept.cpu().double(), act)
    d, hb = B.gated_matmul_backward(x.cuda(), w2.cuda(), gl, kept, **kw)
    _check(d, want, bound, "gradients")
    _check(hb, h_want, h_bound, "h again")


def _calls():
    """Calls on inputs of their own (1 MiB or more each: blocks of their own)."""
    gl = torch.tensor([512, 1024], device="cuda")
    x = torch.randn((1024, 1024), device="cuda").to(BF16)
    w1 = (0.03 * torch.randn((2, 1024, 1024), device="cuda")).to(BF16)
    w2 = (0.03 * torch.randn((2, 512, 1024), device="cuda")).to(BF16)
    _, kept, scale = B.gated_matmul(x, w1, gl, keep="fp8")
    return {
        "forward": (lambda s, x, w: B.gated_matmul(x, w, gl, keep="fp8", stream=s), (x, w1)),
        "backward": (lambda s, dy, w, k, sc: B.gated_matmul_backward(dy, w, gl, k, kept_scale=sc, stream=s), (x, w2, kept, scale)),
        "wgrad": (lambda s, k, sc, dy: (B.grouped_matmul_wgrad(k, dy, gl, x_scale=sc, stream=s),), (kept, scale, x)),
    }


def _bytes(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("name", ["forward", "backward", "wgrad"])
def test_inputs_freed_before_the_side_stream_comes_to_them(name):
    call, inputs = _calls()[name]
    want = call(None, *inputs)
    side = torch.cuda.Stream()
    temporary = [t.clone() for t in inputs]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms in front of the call
    got = call(side, *temporary)
    shapes = [(t.shape, t.dtype) for t in temporary]
    del temporary
    new = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(3)]
    for t in new:
        _bytes(t).fill_(0x7F)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(_bytes(g), _bytes(w)), name
    del new


def test_two_streams_at_once():
    calls = _calls()
    streams = [torch.cuda.Stream() for _ in range(3)]
    want = {n: c(None, *i) for n, (c, i) in calls.items()}
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, (n, (c, i)) in zip(streams, calls.items()):
            got.append((n, c(s, *i)))
    torch.cuda.synchronize()
    for n, outs in got:
        for a, b in zip(outs, want[n]):
            assert torch.equal(_bytes(a), _bytes(b)), n


def test_captured_steps_and_replays():
    """Two graphs of a whole step each, with their own inputs, replayed in turn
    with eager steps of the same between them."""
    rng = np.random.default_rng(12)
    m, e, k, f = 260, 4, 256, 320
    gl = torch.tensor([100, 0, 60, 100]).cuda()
    w1, w2 = _rand(rng, (e, k, 2 * f), scale=0.1).cuda(), _rand(rng, (e, f, k), scale=0.1).cuda()
    ins = [(_rand(rng, (m, k)).cuda(), _rand(rng, (m, k), scale=0.1).cuda()) for _ in range(2)]

    def step(x, dy):
        h, kept, scale = B.gated_matmul(x, w1, gl, keep="fp8", activation="geglu", group_list_type=1)
        codes, xs = B.mx_quantize(x, format="fp8")
        d, hb = B.gated_matmul_backward(dy, w2, gl, kept, kept_scale=scale, activation="geglu", group_list_type=1)
        return (h, d, hb, B.grouped_matmul_wgrad(codes, d, gl, x_scale=xs, group_list_type=1),
                B.grouped_matmul_wgrad(d, codes, gl, dy_scale=xs, group_list_type=1))
    graphs, outs = [], []
    for x, dy in ins:
        step(x, dy)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(x, dy))
        graphs.append(g)
    for turn in range(4):
        for (x, dy), g, got in zip(ins, graphs, outs):
            x.copy_(_rand(rng, (m, k)))
            dy.copy_(_rand(rng, (m, k), scale=0.1))
            for t in got:
                t.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (x, dy), got in zip(ins, outs):
            for a, b in zip(got, step(x, dy)):
                assert torch.equal(a, b), turn


def test_a_training_step_captured_beside_an_eager_one():
    """The Function's forward and backward inside one graph, while an eager
    result of the same leaves is alive."""
    rng = np.random.default_rng(16)
    m, e, k, f = 200, 2, 128, 96
    gl = torch.tensor([80, 120]).cuda()
    leaves = [_rand(rng, s, scale=sc).cuda().requires_grad_() for s, sc in (((m, k), 1.0), ((e, k, 2 * f), 0.1), ((e, f, k), 0.1))]
    dy = _rand(rng, (m, k)).cuda()
    alive = Block.apply(*leaves, gl, "swiglu", "fp8")
    want = torch.autograd.grad(alive, leaves, dy, retain_graph=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(Block.apply(*leaves, gl, "swiglu", "fp8"), leaves, dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        # detached leaves of their own: the eager result's stay out of the capture
        own = [t.detach().requires_grad_() for t in leaves]
        got = torch.autograd.grad(Block.apply(*own, gl, "swiglu", "fp8"), own, dy)
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    for a, b in zip(torch.autograd.grad(alive, leaves, dy), want):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """What is kept, and d, of 4.3e9 elements; rows in FP8 of 2.2e9: sampled."""
    m, e, k, f = 70000, 2, 16, 30720
    gen = torch.Generator(device="cuda").manual_seed(5)

    def normal(*shape, scale=1.0):
        t = torch.empty(shape, dtype=BF16, device="cuda")
        t.normal_(0, scale, generator=gen)
        return t
    x, w1, w2 = normal(m, k), normal(e, k, 2 * f, scale=0.3), normal(e, f, k, scale=0.3)
    gl, ends = torch.tensor([1000, 69000]).cuda(), [1000, 70000]
    rows = [0, 999, 1000, 34952, 34953, 69999]
    wd1, wd2 = w1.cpu().double(), w2.cpu().double()
    for keep in ("fp8", "full"):
        h, kept, scale = B.gated_matmul(x, w1, gl, keep=keep, group_list_type=1)
        d, hb = B.gated_matmul_backward(x, w2, gl, kept, kept_scale=scale, group_list_type=1)
        for i in rows:
            g = 0 if i < ends[0] else 1
            xi = x[i:i + 1].cpu().double()
            both, s = xi @ wd1[g], xi.abs() @ wd1[g].abs() * (k + 1) * R.U
            want, bound = G.forward(both, s, "swiglu")
            _check(h[i:i + 1], want, bound, f"h, row {i}")
            if keep == "fp8":
                values = R.decode(kept[i:i + 1].cpu(), scale[i:i + 1].cpu())
                R.assert_within(values, both, G.fp8_bound(both, s), f"kept, row {i}")
            else:
                values = kept[i:i + 1].cpu().double()
                _check(kept[i:i + 1], both, s, f"kept, row {i}")
            dh, s = xi @ wd2[g].T, xi.abs() @ wd2[g].T.abs() * (k + 1) * R.U
            want, bound, h_want, h_bound = G.backward(dh, s, values, "swiglu")
            _check(d[i:i + 1], want, bound, f"gradients, row {i}")
            _check(hb[i:i + 1], h_want, h_bound, f"h again, row {i}")
        del h, d, hb
        if keep == "fp8":  # 70000 x 61440 codes, the columns of the last rows' group; 16 of the others
            for side in ("x", "dy"):
                a = dict(x_scale=scale) if side == "x" else dict(dy_scale=scale)
                dw = B.grouped_matmul_wgrad(*((kept, x) if side == "x" else (x, kept)), gl, group_list_type=1, **a)
                dw = dw if side == "x" else dw.transpose(1, 2)
                for c in (0, 30719, 61439):
                    col = kept[:, c].float().cpu().double() * torch.exp2(scale.view(torch.uint8).view(m, -1)[:, c // 32].cpu().double() - 127)
                    part = col[1000:, None] * x[1000:].cpu().double()
                    bound = part.abs().sum(0) * 69001 * R.U
                    R.assert_within(dw[1, c], part.sum(0), bound + R.half_step(part.sum(0).abs() + bound, F32), f"dw, column {c}")
                del dw
        del kept, scale


@pytest.mark.parametrize("height", [32, 128, 256])
@pytest.mark.parametrize("transpose", [False, True])
def test_the_largest_sizes(height, transpose):
    """k, d and 2 f of 65536."""
    gen = torch.Generator(device="cuda").manual_seed(6)

    def normal(*shape, scale=1.0):
        t = torch.empty(shape, dtype=BF16, device="cuda")
        t.normal_(0, scale, generator=gen)
        return t
    m, t = 5, [0, height]
    gl = torch.tensor([m]).cuda()
    for k, f in ((65536, 32), (64, 32768)):
        x, w = normal(m, k), normal(1, *((2 * f, k) if transpose else (k, 2 * f)), scale=k ** -0.5)
        h, kept, scale = B.gated_matmul(x, w, gl, keep="fp8", transpose_w=transpose, tuning_config=t)
        wd = (w[0].T if transpose else w[0]).cpu().double()
        both, s = x.cpu().double() @ wd, x.cpu().double().abs() @ wd.abs() * (k + 1) * R.U
        want, bound = G.forward(both, s, "swiglu")
        _check(h, want, bound, "h")
        R.assert_within(R.decode(kept.cpu(), scale.cpu()), both, G.fp8_bound(both, s), "kept")
    for d, f in ((65536, 32), (64, 32768)):
        dy, w, both = normal(m, d), normal(1, *((f, d) if transpose else (d, f)), scale=d ** -0.5), normal(m, 2 * f)
        kept, scale = B.mx_quantize(both, format="fp8")
        got, h = B.gated_matmul_backward(dy, w, gl, kept, kept_scale=scale, transpose_w=transpose, tuning_config=t)
        wd = (w[0].T if transpose else w[0]).cpu().double()
        dh, s = dy.cpu().double() @ wd, dy.cpu().double().abs() @ wd.abs() * (d + 1) * R.U
        want, bound, h_want, h_bound = G.backward(dh, s, R.decode(kept.cpu(), scale.cpu()), "swiglu")
        _check(got, want, bound, "gradients")
        _check(h, h_want, h_bound, "h again")


def test_refusals_on_the_gpu():
    x, w = torch.ones((8, 64), dtype=BF16, device="cuda"), torch.ones((1, 64, 80), dtype=BF16, device="cuda")
    gl = torch.tensor([8]).cuda()
    with pytest.raises(B.GmmfrError, match="SHAPE"):
        B.gated_matmul(x, w, gl, keep="fp8")  # 40 columns are no whole blocks
    with pytest.raises(B.GmmfrError, match="DTYPE"):
        B.gated_matmul(x.float(), w.float(), gl)
    with pytest.raises(ValueError, match="contiguous"):
        B.gated_matmul(x.T.contiguous().T, w, gl)
    with pytest.raises(ValueError, match="device"):
        B.gated_matmul(x, w, gl.cpu())
    h, kept, _ = B.gated_matmul(x, w, gl, keep="full")
    with pytest.raises(B.GmmfrError, match="NULLPTR"):
        B.gated_matmul_backward(x, torch.ones((1, 40, 64), dtype=BF16, device="cuda"), gl, kept.to(torch.float8_e4m3fn))
    with pytest.raises(B.GmmfrError, match="SHAPE"):
        B.gated_matmul_backward(x, torch.ones((1, 64, 40), dtype=BF16, device="cuda"), gl, kept)
    codes, scale = B.mx_quantize(x, format="fp8")
    with pytest.raises(B.GmmfrError, match="DTYPE"):
        B.grouped_matmul_wgrad(codes, x, gl)  # its scales are missing
    with pytest.raises(B.GmmfrError, match="UNSUPPORTED"):
        B.grouped_matmul_wgrad(codes, codes, gl, x_scale=scale, dy_scale=scale)
    with pytest.raises(B.GmmfrError, match="DTYPE"):
        B.grouped_matmul_wgrad(*B.mx_quantize(x, format="fp4")[:1], x, gl, x_scale=scale)


def test_a_calls_status_is_its_own():
    hip = ctypes.CDLL("libamdhip64.so.7")
    gl = torch.tensor([16]).cuda()
    x, w1 = torch.ones((16, 64), dtype=BF16, device="cuda"), torch.ones((1, 64, 64), dtype=BF16, device="cuda")
    h, kept, scale = B.gated_matmul(x, w1, gl, keep="fp8")
    w2, d, dw = torch.ones((1, 32, 64), dtype=BF16, device="cuda"), torch.empty((16, 64), dtype=BF16, device="cuda"), torch.empty((1, 64, 64), device="cuda")
    a, k1 = B.make_gf_args(x, w1, gl, h, kept=kept, kept_scale=scale)
    b, k2 = B.make_gb_args(x, w2, gl, kept, d, kept_scale=scale)
    c, k3 = B.make_gx_args(kept, x, gl, dw, x_scale=scale)
    L, stream = B.lib(), torch.cuda.current_stream().cuda_stream
    for name, args in (("gmm_gated_matmul", a), ("gmm_gated_matmul_backward", b), ("gmm_grouped_matmul_wgrad_fp8", c)):
        torch.cuda.synchronize()
        hip.hipGetLastError()
        status = hip.hipSetDevice(9999)
        assert status != 0
        assert getattr(L, name)(ctypes.byref(args), None, 0, stream) == B.OK, name
        assert hip.hipGetLastError() == status, name
    torch.cuda.synchronize()
