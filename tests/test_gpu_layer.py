"""The new operators as a layer uses them, together with the ones that were
there: the producer step's MX modes, the gate and up projections with SwiGLU,
requantisation and the combining product; and a training step's three products."""
import numpy as np
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu


def _route(rng, tokens, top, experts):
    ids = np.stack([rng.permutation(experts)[:top] for _ in range(tokens)])
    w = rng.random((tokens, top)).astype(np.float32)
    return torch.from_numpy(ids), torch.from_numpy(w)


@pytest.mark.parametrize("mode", ["mx", "mx4"])
@pytest.mark.parametrize("tokens,k,f,n,local,offset", [(37, 320, 192, 352, 5, 2), (1, 512, 128, 256, 8, 0),
                                                       (300, 1088, 576, 544, 4, 1)])
def test_microscaled_layer(mode, tokens, k, f, n, local, offset):
    """Each stage against the 64-bit form of what the stage before it gave."""
    rng = np.random.default_rng(tokens)
    top, experts = 3, 8
    hidden = torch.from_numpy(rng.standard_normal((tokens, k)) * np.exp(rng.standard_normal(k))).bfloat16().cuda()
    ids, weights = _route(rng, tokens, top, experts)
    w13 = torch.from_numpy(rng.standard_normal((local, k, 2 * f)) * k ** -0.5).bfloat16().cuda()
    w2 = torch.from_numpy(rng.standard_normal((local, n, f)) * f ** -0.5).bfloat16().cuda()
    c13, s13 = B.mx_quantize(w13, transpose=True)   # as stored (e,k,n), brought to (e,n,k)
    c2, s2 = B.mx_quantize(w2)
    qp = B.quant_permute(hidden, ids.cuda(), local, topk_weights=weights.cuda(), expert_offset=offset, mode=mode)
    act = B.grouped_matmul(qp["x1"], c13, qp["group_list"], x_scale=qp["pertoken_scale"], w_scale=s13, transpose_w=True,
                           activation="swiglu", group_list_type=1)
    a8, as8 = B.mx_quantize(act, format="fp8")
    out = torch.empty((tokens, n), dtype=torch.float32, device="cuda")
    B.gmm_finalize_routing(a8, c2, qp["group_list"], out, scale=s2, pertoken_scale=as8, logit=qp["logit"],
                           row_index=qp["row_index"], group_list_type=1, deterministic=True, transpose_x2=True)
    torch.cuda.synchronize()

    counts = qp["group_list"].cpu().numpy()
    rows = int(counts.sum())
    assert rows == int(((ids >= offset) & (ids < offset + local)).sum())
    token = qp["row_index"].cpu()[:rows]
    # the producer step's codes: those of mx_quantize on the tokens' rows
    fmt = "fp8" if mode == "mx" else "fp4"
    codes, scales = B.mx_quantize(hidden, format=fmt)
    assert torch.equal(qp["x1"].view(torch.uint8).cpu()[:rows], codes.view(torch.uint8).cpu()[token])
    assert torch.equal(qp["pertoken_scale"].view(torch.uint8).cpu()[:rows], scales.view(torch.uint8).cpu()[token])

    def host(t):
        return t.cpu()
    x1, pts = qp["x1"].view(torch.uint8).cpu()[:rows].view(qp["x1"].dtype), host(qp["pertoken_scale"])[:rows]
    x, w = R.decode(x1, pts), R.decode(host(c13), host(s13))
    want, s = R.product(x, w.transpose(1, 2), counts, 1)
    err = s * (k // 32 + 32) * R.U
    if mode == "mx":
        for g, (a, b) in enumerate(R.groups(counts, rows, 1)):
            if b > a:
                err[a:b] += R.mx_block_loss(R.elements(x1[a:b]), R.scale_values(pts[a:b]), R.elements(host(c13)[g]),
                                            R.scale_values(host(s13)[g]))
    want, err = R.swiglu(want, err)
    R.assert_within(act[:rows], want, err + R.half_step(want.abs() + err, torch.bfloat16), "activation")

    # the requantised rows, then the combine
    cc, ss = R.encode(act[:rows].float().cpu().numpy(), "fp8")
    pc, ps = R.pack(cc, ss, "fp8")
    assert torch.equal(pc.view(torch.uint8), a8.view(torch.uint8).cpu()[:rows])
    assert torch.equal(ps.view(torch.uint8), as8.view(torch.uint8).cpu()[:rows])
    h, v = R.decode(pc, ps), R.decode(host(c2), host(s2))
    y, s = R.product(h, v.transpose(1, 2), counts, 1)
    err = s * (f // 32 + 32) * R.U
    for g, (a, b) in enumerate(R.groups(counts, rows, 1)):
        if b > a:
            err[a:b] += R.mx_block_loss(R.elements(pc[a:b]), R.scale_values(ps[a:b]), R.elements(host(c2)[g]),
                                        R.scale_values(host(s2)[g]))
    lg = qp["logit"].cpu().double()[:rows, None]
    ref = torch.zeros((tokens, n), dtype=torch.float64).index_add_(0, token, y * lg)
    bound = torch.zeros((tokens, n), dtype=torch.float64).index_add_(0, token, (err + y.abs() * (top + 2) * R.U) * lg.abs())
    R.assert_within(out, ref, bound + 1e-37, "combined")


def test_training_step_of_the_products():
    """y, dx and dw of one grouped product against automatic differentiation in
    64 bits on the same bf16 inputs, and dw summed over two steps."""
    rng = np.random.default_rng(3)
    m, e, k, n = 400, 5, 192, 264
    counts = R.counts_for(rng, m, e, 0.2)
    gl = torch.from_numpy(counts)
    x = torch.from_numpy(rng.standard_normal((m, k))).bfloat16()
    w = torch.from_numpy(rng.standard_normal((e, k, n)) * k ** -0.5).bfloat16()
    dy = torch.from_numpy(rng.standard_normal((m, n))).bfloat16()
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    ends = np.cumsum(counts)
    y = torch.cat([xd[b - c:b] @ wd[g] for g, (b, c) in enumerate(zip(ends, counts))])
    y.backward(dy.double())
    d = gl.cuda()
    got = B.grouped_matmul(x.cuda(), w.cuda(), d, group_list_type=1)
    dx = B.grouped_matmul(dy.cuda(), w.cuda(), d, transpose_w=True, group_list_type=1)
    dw = B.grouped_matmul_wgrad(x.cuda(), dy.cuda(), d, group_list_type=1)

    def check(a, want, s, terms, dtype, what):
        bound = s * (terms + 1) * R.U
        R.assert_within(a, want, bound + R.half_step(want.abs() + bound, dtype), what)
    _, s = R.product(x.double(), w.double(), counts, 1)
    check(got, y.detach(), s, k, torch.bfloat16, "y")
    _, s = R.product(dy.double(), w.double().transpose(1, 2), counts, 1)
    check(dx, xd.grad, s, n, torch.bfloat16, "dx")
    _, s, rows = R.wgrad(x.double(), dy.double(), counts, 1)
    check(dw, wd.grad, s, rows[:, None, None], torch.float32, "dw")
    B.grouped_matmul_wgrad(x.cuda(), dy.cuda(), d, out=dw, accumulate=True, group_list_type=1)
    check(dw, 2 * wd.grad, 2 * s, rows[:, None, None] + 1, torch.float32, "dw of two steps")


def test_two_streams_at_once():
    """Two calls that overlap on one GPU share nothing."""
    rng = np.random.default_rng(4)
    m, e, k, n = 3000, 6, 512, 1024
    gl = R.as_list(R.counts_for(rng, m, e), 1).cuda()
    xs = [torch.from_numpy(rng.standard_normal((m, k))).bfloat16().cuda() for _ in range(2)]
    w = torch.from_numpy(rng.standard_normal((e, k, n))).bfloat16().cuda()
    want = [B.grouped_matmul(x, w, gl, group_list_type=1) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i in (0, 1):
            got[i].append(B.grouped_matmul(xs[i], w, gl, group_list_type=1, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for y in got[i]:
            assert torch.equal(y, want[i])
