"""Stage one of the gated block and of its way back on the CPU: every refusal,
and what is accepted (fake pointers, never dereferenced; nothing is launched)."""
import ctypes

import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests.test_boundary_grouped import BF, E8, F16, F32, FP4, FP8, I64, fake, gm, put, stage_one

NONE = B.Tensor()


def gf(m=300, k=512, f=192, e=4, dt=BF, **over):
    a = B.GfArgs()
    a.x, a.w, a.group_list, a.h, a.activation = fake(dt, m, k), fake(dt, e, k, 2 * f), fake(I64, e), fake(dt, m, f), 1
    return put(a, over)


def gb(m=300, k=512, f=192, e=4, dt=BF, **over):
    a = B.GbArgs()
    a.dy, a.w, a.group_list, a.kept = fake(dt, m, k), fake(dt, e, f, k), fake(I64, e), fake(dt, m, 2 * f)
    a.d, a.h, a.transpose_w, a.activation = fake(dt, m, 2 * f), fake(dt, m, f), 1, 1
    return put(a, over)


def in_fp8(m=300, f=192):
    return dict(kept=fake(FP8, m, 2 * f), kept_scale=fake(E8, m, 2 * f // 64, 2))


CASES = [
    (gf, {}, B.OK), (gf, dict(dt=F16), B.OK), (gf, dict(activation=2), B.OK), (gf, dict(m=0), B.OK),
    (gf, dict(kept=fake(BF, 300, 384)), B.OK), (gf, in_fp8(), B.OK),
    (gf, dict(f=40), B.OK), (gf, dict(k=8, f=8), B.OK), (gf, dict(e=1024), B.OK),
    (gf, dict(transpose_w=1, w=fake(BF, 4, 384, 512)), B.OK),
    (gf, dict(tuning=[7, 256, 3]), B.OK),
    (gb, {}, B.OK), (gb, dict(dt=F16), B.OK), (gb, dict(activation=2, m=0), B.OK), (gb, in_fp8(), B.OK),
    (gb, dict(h=NONE), B.OK), (gb, dict(f=40), B.OK), (gb, dict(transpose_w=0, w=fake(BF, 4, 512, 192)), B.OK),
    (gf, dict(x=NONE), B.ERR_NULLPTR), (gf, dict(w=NONE), B.ERR_NULLPTR), (gf, dict(group_list=NONE), B.ERR_NULLPTR),
    (gf, dict(h=NONE), B.ERR_NULLPTR), (gf, dict(kept=fake(FP8, 300, 384)), B.ERR_NULLPTR),
    (gf, dict(kept_scale=fake(E8, 300, 6, 2)), B.ERR_NULLPTR),
    (gb, dict(dy=NONE), B.ERR_NULLPTR), (gb, dict(w=NONE), B.ERR_NULLPTR), (gb, dict(group_list=NONE), B.ERR_NULLPTR),
    (gb, dict(kept=NONE), B.ERR_NULLPTR), (gb, dict(d=NONE), B.ERR_NULLPTR),
    (gb, dict(kept=fake(FP8, 300, 384)), B.ERR_NULLPTR),
    (gf, dict(dt=F32), B.ERR_DTYPE), (gf, dict(x=fake(FP8, 300, 512)), B.ERR_DTYPE), (gf, dict(w=fake(F16, 4, 512, 384)), B.ERR_DTYPE),
    (gf, dict(h=fake(F32, 300, 192)), B.ERR_DTYPE), (gf, dict(kept=fake(F16, 300, 384)), B.ERR_DTYPE),
    (gf, dict(kept=fake(FP4, 300, 192)), B.ERR_DTYPE), (gf, dict(kept=fake(FP8, 300, 384), kept_scale=fake(F32, 300, 6, 2)), B.ERR_DTYPE),
    (gf, dict(group_list=fake(B.DT_INT32, 4)), B.ERR_DTYPE),
    (gb, dict(dt=F32), B.ERR_DTYPE), (gb, dict(d=fake(F32, 300, 384)), B.ERR_DTYPE), (gb, dict(h=fake(F16, 300, 192)), B.ERR_DTYPE),
    (gb, dict(kept=fake(F32, 300, 384)), B.ERR_DTYPE), (gb, dict(w=fake(F16, 4, 192, 512)), B.ERR_DTYPE),
    (gf, dict(kept=fake(BF, 300, 384), kept_scale=fake(E8, 300, 6, 2)), B.ERR_UNSUPPORTED),
    (gb, dict(kept_scale=fake(E8, 300, 6, 2)), B.ERR_UNSUPPORTED),
    (gf, dict(activation=0), B.ERR_ATTR), (gf, dict(activation=3), B.ERR_ATTR), (gf, dict(transpose_w=2), B.ERR_ATTR),
    (gf, dict(group_list_type=2), B.ERR_ATTR), (gf, dict(tuning=[0, 64]), B.ERR_ATTR), (gf, dict(tuning_config_len=1), B.ERR_ATTR),
    (gb, dict(activation=0), B.ERR_ATTR), (gb, dict(transpose_w=-1), B.ERR_ATTR), (gb, dict(group_list_type=-1), B.ERR_ATTR),
    (gb, dict(tuning=[-1]), B.ERR_ATTR),
    (gf, dict(k=516), B.ERR_SHAPE), (gf, dict(f=36), B.ERR_SHAPE), (gf, dict(f=40, **in_fp8(300, 40)), B.ERR_SHAPE),
    (gf, dict(e=1025), B.ERR_SHAPE), (gf, dict(h=fake(BF, 300, 384)), B.ERR_SHAPE), (gf, dict(h=fake(BF, 299, 192)), B.ERR_SHAPE),
    (gf, dict(kept=fake(BF, 300, 192)), B.ERR_SHAPE), (gf, dict(kept=fake(FP8, 300, 384), kept_scale=fake(E8, 300, 12)), B.ERR_SHAPE),
    (gf, dict(w=fake(BF, 4, 384, 512)), B.ERR_SHAPE), (gf, dict(group_list=fake(I64, 3)), B.ERR_SHAPE),
    (gf, dict(k=65536, f=32768, transpose_w=1, w=fake(BF, 4, 65536, 65536)), B.ERR_SHAPE),
    (gb, dict(d=fake(BF, 300, 192)), B.ERR_SHAPE), (gb, dict(d=fake(BF, 300, 383)), B.ERR_SHAPE), (gb, dict(h=fake(BF, 300, 384)), B.ERR_SHAPE),
    (gb, dict(kept=fake(BF, 301, 384)), B.ERR_SHAPE), (gb, dict(f=36), B.ERR_SHAPE), (gb, dict(d=fake(BF, 300, 384, 1)), B.ERR_SHAPE),
    (gf, dict(f=32768, k=8), B.OK), (gb, dict(f=32768, k=8), B.OK), (gf, dict(f=32776, k=8), B.ERR_SHAPE), (gb, dict(f=32776, k=8), B.ERR_SHAPE),
    (gb, dict(transpose_w=0), B.ERR_SHAPE), (gb, dict(f=40, **in_fp8(300, 40)), B.ERR_SHAPE),
    (gf, dict(h=fake(BF, 300, 192, ptr=0x7000008)), B.ERR_ALIGN), (gf, dict(kept=fake(BF, 300, 384, ptr=0x7000002)), B.ERR_ALIGN),
    (gb, dict(h=fake(BF, 300, 192, ptr=0x7000008)), B.ERR_ALIGN), (gb, dict(kept=fake(BF, 300, 384, ptr=0x7000002)), B.ERR_ALIGN),
    (gb, dict(kept=fake(FP8, 300, 384), kept_scale=fake(E8, 300, 6, 2, ptr=0x7000004)), B.ERR_ALIGN),
]


@pytest.mark.parametrize("make,over,code", CASES, ids=[str(i) for i in range(len(CASES))])
def test_stage_one(make, over, code):
    sizes = {k: v for k, v in over.items() if k in ("m", "k", "f", "e", "dt")}
    a = make(**sizes, **{k: v for k, v in over.items() if k not in sizes})
    name = "gmm_gated_matmul" if make is gf else "gmm_gated_matmul_backward"
    assert stage_one(name, a) == (code, 0 if code == B.OK else 12345)
    if code != B.OK:  # before any launch
        assert getattr(B.lib(), name)(ctypes.byref(a), None, 0, None) == code


@pytest.mark.parametrize("name,make", [("gmm_gated_matmul", gf), ("gmm_gated_matmul_backward", gb)])
def test_null_pointers_and_no_rows(name, make):
    assert getattr(B.lib(), name + "_workspace")(None, ctypes.byref(ctypes.c_size_t())) == B.ERR_NULLPTR
    assert getattr(B.lib(), name + "_workspace")(ctypes.byref(make()), None) == B.ERR_NULLPTR
    assert getattr(B.lib(), name)(None, None, 0, None) == B.ERR_NULLPTR
    assert getattr(B.lib(), name)(ctypes.byref(make(m=0)), None, 0, None) == B.OK  # nothing to launch


def _tensors():
    bf = torch.bfloat16
    return dict(x=torch.zeros((8, 64), dtype=bf), w=torch.zeros((2, 64, 64), dtype=bf), gl=torch.tensor([4, 8]),
                dy=torch.zeros((8, 16), dtype=bf), wd=torch.zeros((2, 32, 16), dtype=bf), kept=torch.zeros((8, 64), dtype=bf))


def test_packed_descriptors_are_the_structs():
    t = _tensors()
    h = torch.zeros((8, 32), dtype=torch.bfloat16)
    a, _ = B.make_gf_args(t["x"], t["w"], t["gl"], h, kept=t["kept"], group_list_type=1, activation="geglu", tuning_config=[5, 32])
    for name, v in (("x", t["x"]), ("w", t["w"]), ("group_list", t["gl"]), ("h", h), ("kept", t["kept"]), ("kept_scale", None)):
        d, want = getattr(a, name), B._desc(v)
        assert (d.data, d.dtype, d.ndim, list(d.dims)) == (want.data, want.dtype, want.ndim, list(want.dims))
    assert (a.group_list_type, a.transpose_w, a.activation, list(a.tuning_config[:2])) == (1, 0, 2, [5, 32])
    b, _ = B.make_gb_args(t["dy"], t["wd"], t["gl"], t["kept"], t["x"], h=h)
    for name, v in (("dy", t["dy"]), ("w", t["wd"]), ("group_list", t["gl"]), ("kept", t["kept"]), ("kept_scale", None),
                    ("d", t["x"]), ("h", h)):
        d, want = getattr(b, name), B._desc(v)
        assert (d.data, d.dtype, d.ndim, list(d.dims)) == (want.data, want.dtype, want.ndim, list(want.dims))
    assert (b.group_list_type, b.transpose_w, b.activation, bool(b.tuning_config)) == (0, 1, 1, False)


def test_python_entry_refuses():
    t = _tensors()
    with pytest.raises(ValueError, match="GPU"):
        B.gated_matmul(t["x"], t["w"], t["gl"])
    with pytest.raises(ValueError, match="GPU"):
        B.gated_matmul_backward(t["dy"], t["wd"], t["gl"], t["kept"])
    with pytest.raises(ValueError, match="activation"):
        B.gated_matmul(t["x"], t["w"], t["gl"], activation="relu")
    with pytest.raises(ValueError, match="activation"):
        B.gated_matmul_backward(t["dy"], t["wd"], t["gl"], t["kept"], activation=None)
    with pytest.raises(ValueError, match="keep"):
        B.gated_matmul(t["x"], t["w"], t["gl"], keep="int8")
    with pytest.raises(ValueError, match="keep"):
        B.gated_matmul(t["x"], t["w"], t["gl"], kept=t["kept"])
    with pytest.raises(ValueError, match="keep"):
        B.gated_matmul(t["x"], t["w"], t["gl"], keep="full", kept_scale=t["kept"])
    with pytest.raises(ValueError, match="wanted"):
        B.gated_matmul_backward(t["dy"], t["wd"], t["gl"], t["kept"], h=t["x"], want_h=False)


@pytest.mark.parametrize("which", ["x", "w", "dy", "wd", "kept"])
def test_a_lost_gradient_is_refused(which):
    t = _tensors()
    t[which].requires_grad_()
    calls = [lambda: B.gated_matmul(t["x"], t["w"], t["gl"])] if which in "xw" else \
            [lambda: B.gated_matmul_backward(t["dy"], t["wd"], t["gl"], t["kept"])]
    for call in calls:
        with pytest.raises(ValueError, match="no_grad"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            call()


def gx(m=300, k=512, n=384, e=4, dt=BF, side="x", **over):
    a = B.GxArgs()
    a.x, a.dy, a.group_list, a.dw = fake(dt, m, k), fake(dt, m, n), fake(I64, e), fake(F32, e, k, n)
    if side == "x":
        a.x, a.x_scale = fake(FP8, m, k), fake(E8, m, k // 64, 2)
    else:
        a.dy, a.dy_scale = fake(FP8, m, n), fake(E8, m, n // 64, 2)
    return put(a, over)


GX_CASES = [
    ({}, B.OK), (dict(side="dy"), B.OK), (dict(dt=F16), B.OK), (dict(m=0), B.OK), (dict(accumulate=1), B.OK), (dict(n=8), B.OK),
    (dict(side="dy", k=8), B.OK), (dict(dw=fake(BF, 4, 512, 384)), B.OK), (dict(tuning=[0, 128, 4]), B.OK),
    (dict(x=NONE), B.ERR_NULLPTR), (dict(dy=NONE), B.ERR_NULLPTR), (dict(dw=NONE), B.ERR_NULLPTR), (dict(group_list=NONE), B.ERR_NULLPTR),
    (dict(x_scale=NONE), B.ERR_NULLPTR), (dict(side="dy", dy_scale=NONE), B.ERR_NULLPTR),
    (dict(x=fake(BF, 300, 512)), B.ERR_DTYPE), (dict(dy=fake(FP8, 300, 384)), B.ERR_DTYPE), (dict(dt=F32), B.ERR_DTYPE),
    (dict(x=fake(FP4, 300, 256)), B.ERR_DTYPE), (dict(x_scale=fake(F32, 300, 8, 2)), B.ERR_DTYPE), (dict(dw=fake(F16, 4, 512, 384)), B.ERR_DTYPE),
    (dict(dy_scale=fake(E8, 300, 6, 2)), B.ERR_UNSUPPORTED), (dict(side="dy", x_scale=fake(E8, 300, 8, 2)), B.ERR_UNSUPPORTED),
    (dict(accumulate=2), B.ERR_ATTR), (dict(accumulate=1, dw=fake(BF, 4, 512, 384)), B.ERR_ATTR), (dict(group_list_type=3), B.ERR_ATTR),
    (dict(tuning=[0, 32]), B.ERR_ATTR),
    (dict(k=520), B.ERR_SHAPE), (dict(side="dy", n=392), B.ERR_SHAPE), (dict(n=12), B.ERR_SHAPE), (dict(x_scale=fake(E8, 300, 16)), B.ERR_SHAPE),
    (dict(x_scale=fake(E8, 299, 8, 2)), B.ERR_SHAPE), (dict(e=1025), B.ERR_SHAPE), (dict(dw=fake(F32, 4, 384, 512)), B.ERR_SHAPE),
    (dict(x=fake(FP8, 300, 512, ptr=0x7000008)), B.ERR_ALIGN), (dict(x_scale=fake(E8, 300, 8, 2, ptr=0x7000002)), B.ERR_ALIGN),
]


@pytest.mark.parametrize("over,code", GX_CASES, ids=[str(i) for i in range(len(GX_CASES))])
def test_wgrad_fp8_stage_one(over, code):
    sizes = {k: v for k, v in over.items() if k in ("m", "k", "n", "e", "dt", "side")}
    a = gx(**sizes, **{k: v for k, v in over.items() if k not in sizes})
    assert stage_one("gmm_grouped_matmul_wgrad_fp8", a) == (code, 0 if code == B.OK else 12345)
    if code != B.OK:
        assert B.lib().gmm_grouped_matmul_wgrad_fp8(ctypes.byref(a), None, 0, None) == code


def test_wgrad_fp8_null_pointers():
    L, a = B.lib(), gx()
    assert L.gmm_grouped_matmul_wgrad_fp8_workspace(None, ctypes.byref(ctypes.c_size_t())) == B.ERR_NULLPTR
    assert L.gmm_grouped_matmul_wgrad_fp8_workspace(ctypes.byref(a), None) == B.ERR_NULLPTR
    assert L.gmm_grouped_matmul_wgrad_fp8(None, None, 0, None) == B.ERR_NULLPTR


@pytest.mark.parametrize("n,tile", [(4096, 256), (2048, 128)])
def test_one_experts_rows_are_whole_tiles(n, tile):
    """4096 rows are 16 tiles of 256: with 4096 columns one round of the chip,
    with 2048 half a round, where 128-row tiles make a whole one."""
    for rows in ([], [4096], [0]):
        assert B.gm_plan(gm(m=4096, k=7168, n=n, e=1, **(dict(tuning=rows) if rows else {})))["tile_m"] == tile


@pytest.mark.parametrize("sizes,parts", [
    (dict(m=2047, k=128, n=128, e=1), 0), (dict(m=2048, k=128, n=128, e=1), 2), (dict(m=40000, k=128, n=128, e=1), 16),
    (dict(m=40000, k=128, n=128, e=20), 0), (dict(m=40960, k=1024, n=4096, e=1), 4), (dict(m=40960, k=2048, n=4096, e=1), 2), (dict(m=40960, k=4096, n=4096, e=1), 0),
])
def test_wgrad_fp8_workspace(sizes, parts):
    """Long groups under few tiles are split: a workspace of fp32 results a part."""
    a = gx(**sizes)
    need = parts * 4 * sizes["e"] * sizes["k"] * sizes["n"]
    assert stage_one("gmm_grouped_matmul_wgrad_fp8", a) == (B.OK, need)
    if need:  # refused before any launch
        call = B.lib().gmm_grouped_matmul_wgrad_fp8
        assert call(ctypes.byref(a), None, 0, None) == B.ERR_WORKSPACE
        assert call(ctypes.byref(a), ctypes.c_void_p(0x10000), need - 1, None) == B.ERR_WORKSPACE
        assert call(ctypes.byref(a), ctypes.c_void_p(0x10008), need, None) == B.ERR_ALIGN
