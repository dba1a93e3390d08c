"""The weight gradient of FP8 rows where the plan splits the groups' rows: the
parts' sums met in a workspace."""
import ctypes

import numpy as np
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _inputs(seed, m, k, n, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((m, k), generator=gen, device="cuda")
    codes, scale = B.mx_quantize(x, format="fp8")
    return codes, scale, (0.1 * torch.randn((m, n), generator=gen, device="cuda")).to(dtype)


def _need(codes, scale, other, gl, dw, side, **kw):
    a, keep = B.make_gx_args(*((codes, other) if side == "x" else (other, codes)), gl, dw,
                             **{("x_scale" if side == "x" else "dy_scale"): scale}, **kw)
    n = ctypes.c_size_t(1)
    assert B.lib().gmm_grouped_matmul_wgrad_fp8_workspace(ctypes.byref(a), ctypes.byref(n)) == B.OK
    del keep
    return n.value


def _call(codes, scale, other, gl, side, **kw):
    if side == "x":
        return B.grouped_matmul_wgrad(codes, other, gl, x_scale=scale, **kw)
    return B.grouped_matmul_wgrad(other, codes, gl, dy_scale=scale, **kw)


@pytest.mark.parametrize("height", [0, 128, 256])
@pytest.mark.parametrize("side", ["x", "dy"])
@pytest.mark.parametrize("counts,k,n,dtype,out", [
    ([9000], 320, 200, BF16, F32),
    ([7000, 0, 100, 1333], 192, 72, F16, F16),   # parts that end inside a step, and beyond short groups
    ([4096, 4097], 448, 264, BF16, BF16),
    ([33, 5, 20000 - 38], 64, 8, F16, F32),
])
def test_split_groups(height, side, counts, k, n, dtype, out):
    m, e = sum(counts) + 3, len(counts)
    codes, scale, other = _inputs(k, m, k, n, dtype)
    scale.view(torch.uint8)[m - 3:] = 255
    other[m - 3:] = float("nan")
    gl = torch.tensor(counts).cuda()
    kw = dict(group_list_type=1, tuning_config=[0, height])
    dw = torch.empty((e, k, n) if side == "x" else (e, n, k), dtype=out, device="cuda")
    need = _need(codes, scale, other, gl, dw, side, **kw)
    assert need and need % (4 * e * k * n) == 0 and 2 <= need // (4 * e * k * n) <= 16
    workspace = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN: it needs no initialisation
    got = _call(codes, scale, other, gl, side, out=dw, workspace=workspace, **kw)
    assert got is dw
    x = B.mx_dequantize(codes[:m - 3].contiguous(), scale[:m - 3].contiguous(), dtype=dtype).double().cpu()
    y = other[:m - 3].double().cpu()
    want, size, rows = R.wgrad(*((x, y) if side == "x" else (y, x)), counts, 1)
    bound = size * (rows + 1)[:, None, None] * R.U
    R.assert_within(got, want, bound + R.half_step(want.abs() + bound, out), "dw")
    # sums this long are off by far less than that bound: of the norm, a few 2^-24 of fp32, or the rounding
    assert float((got.double().cpu() - want).norm() / want.norm()) <= (2.0 ** -18 if out == F32 else torch.finfo(out).eps)
    # the same again, with a workspace of the call's own, and under any grid
    assert torch.equal(_call(codes, scale, other, gl, side, out_dtype=out, **kw), got)
    for cap in (1, 9, 100):
        assert torch.equal(_call(codes, scale, other, gl, side, out_dtype=out, group_list_type=1, tuning_config=[0, height, cap]), got)
    if out == F32:
        before = torch.randn(got.shape, device="cuda")
        assert torch.equal(_call(codes, scale, other, gl, side, out=before.clone(), accumulate=True, **kw), before + got)


@pytest.mark.parametrize("list_type,gl", [(0, [5000, 3000, 9000]), (0, [-5, 4000, 50000]), (1, [3000, -9, 6000]), (1, [8000, 8000, 8000]), (1, [0, 0, 0])])
def test_broken_group_lists(list_type, gl):
    m, k, n = 10000, 64, 72
    codes, scale, other = _inputs(3, m, k, n, BF16)
    got = B.grouped_matmul_wgrad(codes, other, torch.tensor(gl).cuda(), x_scale=scale, group_list_type=list_type)
    want, size, rows = R.wgrad(B.mx_dequantize(codes, scale).double().cpu(), other.double().cpu(), gl, list_type)
    bound = size * (rows + 1)[:, None, None] * R.U
    R.assert_within(got, want, bound + R.half_step(want.abs() + bound, F32), "dw")


def test_two_graphs_and_a_side_stream():
    m, k, n = 9000, 192, 136
    gl = torch.tensor([9000]).cuda()
    sets = [_inputs(s, m, k, n, BF16) for s in (1, 2)]
    graphs, outs = [], []
    for c, s, o in sets:
        B.grouped_matmul_wgrad(c, o, gl, x_scale=s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(B.grouped_matmul_wgrad(c, o, gl, x_scale=s))
        graphs.append(g)
    side = torch.cuda.Stream()
    for turn in range(3):
        for (c, s, o), out in zip(sets, outs):
            o.copy_(torch.randn_like(o))
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (c, s, o), out in zip(sets, outs):
            want = B.grouped_matmul_wgrad(c, o, gl, x_scale=s)
            other = B.grouped_matmul_wgrad(c, o, gl, x_scale=s, stream=side)
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(other, want), turn


def test_a_workspace_too_small_is_refused():
    codes, scale, other = _inputs(4, 9000, 64, 64, BF16)
    gl = torch.tensor([9000]).cuda()
    with pytest.raises(B.GmmfrError, match="WORKSPACE"):
        B.grouped_matmul_wgrad(codes, other, gl, x_scale=scale, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
