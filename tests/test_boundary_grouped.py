"""Stage one of the grouped products, the weight gradient and the MX
quantisation on the CPU: every refusal, and what is accepted (pointers here are
fake, aligned, never dereferenced; nothing is launched)."""
import ctypes

import pytest
import torch

from quantized_moe_grouped_amd import binding as B

_next = [0x10000]


def fake(dtype, *dims, ptr=None):
    t = B.Tensor()
    if ptr is None:
        _next[0] += 0x100000
        ptr = _next[0]
    t.data, t.dtype, t.ndim = ptr, dtype, len(dims)
    for i, d in enumerate(dims):
        t.dims[i] = d
    return t


def stage_one(name, a):
    n = ctypes.c_size_t(12345)
    st = getattr(B.lib(), name + "_workspace")(ctypes.byref(a), ctypes.byref(n))
    return st, n.value


def put(a, over):
    for key, v in over.items():
        if key == "tuning":
            arr = (ctypes.c_int64 * len(v))(*v)
            a.tuning_config = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int64))
            a.tuning_config_len = len(v)
            a.keep = arr
        else:
            setattr(a, key, v)
    return a


BF, F16, F32, I64 = B.DT_BFLOAT16, B.DT_FLOAT16, B.DT_FLOAT32, B.DT_INT64
FP4, FP8, E8 = B.DT_FLOAT4_E2M1X2, B.DT_FLOAT8_E4M3FN, B.DT_FLOAT8_E8M0


def gm(m=300, k=512, n=384, e=4, dt=BF, **over):
    a = B.GmArgs()
    a.x, a.w, a.group_list, a.y = fake(dt, m, k), fake(dt, e, k, n), fake(I64, e), fake(dt, m, n)
    return put(a, over)


def mx(m=300, k=512, n=384, e=4, xt=FP4, **over):
    a = B.GmArgs()
    a.x = fake(xt, m, k // 2 if xt == FP4 else k)
    a.w, a.group_list, a.y = fake(FP4, e, n, k // 2), fake(I64, e), fake(BF, m, n)
    a.x_scale, a.w_scale = fake(E8, m, k // 64, 2), fake(E8, e, n, k // 64, 2)
    a.transpose_w = 1
    return put(a, over)


def gw(m=300, k=512, n=384, e=4, dt=BF, **over):
    a = B.GwArgs()
    a.x, a.dy, a.group_list, a.dw = fake(dt, m, k), fake(dt, m, n), fake(I64, e), fake(F32, e, k, n)
    return put(a, over)


GM_CASES = [
    (gm, {}, B.OK), (mx, {}, B.OK), (mx, dict(xt=FP8), B.OK), (gm, dict(dt=F16), B.OK),
    (gm, dict(y=fake(F32, 300, 384)), B.OK),
    (gm, dict(m=0), B.OK),
    (gm, dict(k=8, n=8), B.OK),
    (gm, dict(transpose_w=1, w=fake(BF, 4, 384, 512)), B.OK),
    (gm, dict(activation=1, y=fake(BF, 300, 192)), B.OK),
    (mx, dict(y=fake(F16, 300, 384)), B.OK),
    (gm, dict(tuning=[7, 256, 3]), B.OK),
    (gm, dict(x=B.Tensor()), B.ERR_NULLPTR),
    (gm, dict(group_list=B.Tensor()), B.ERR_NULLPTR),
    (gm, dict(y=B.Tensor()), B.ERR_NULLPTR),
    (mx, dict(x_scale=B.Tensor()), B.ERR_NULLPTR),
    (mx, dict(w_scale=B.Tensor()), B.ERR_NULLPTR),
    (gm, dict(x=fake(F32, 300, 512)), B.ERR_DTYPE),
    (gm, dict(w=fake(F16, 4, 512, 384)), B.ERR_DTYPE),
    (gm, dict(y=fake(F16, 300, 384)), B.ERR_DTYPE),
    (gm, dict(group_list=fake(B.DT_INT32, 4)), B.ERR_DTYPE),
    (mx, dict(w=fake(FP8, 4, 384, 512)), B.ERR_DTYPE),
    (mx, dict(x_scale=fake(F32, 300, 8, 2)), B.ERR_DTYPE),
    (mx, dict(y=fake(FP8, 300, 384)), B.ERR_DTYPE),
    (gm, dict(x_scale=fake(E8, 300, 8, 2)), B.ERR_UNSUPPORTED),
    (gm, dict(group_list_type=2), B.ERR_ATTR),
    (gm, dict(transpose_w=2), B.ERR_ATTR),
    (mx, dict(transpose_w=0), B.ERR_ATTR),
    (gm, dict(activation=2), B.ERR_ATTR),
    (gm, dict(tuning=[0, 64]), B.ERR_ATTR),
    (gm, dict(tuning=[-1]), B.ERR_ATTR),
    (gm, dict(tuning=[0, 0, -1]), B.ERR_ATTR),
    (gm, dict(tuning_config_len=1), B.ERR_ATTR),
    (gm, dict(tuning_config_len=-1), B.ERR_ATTR),
    (gm, dict(k=516), B.ERR_SHAPE),
    (gm, dict(n=388), B.ERR_SHAPE),
    (gm, dict(k=65544), B.ERR_SHAPE),
    (gm, dict(n=65544), B.ERR_SHAPE),
    (gm, dict(e=1025), B.ERR_SHAPE),
    (gm, dict(w=fake(BF, 4, 520, 384)), B.ERR_SHAPE),
    (gm, dict(w=fake(BF, 512, 384)), B.ERR_SHAPE),
    (gm, dict(transpose_w=1), B.ERR_SHAPE),
    (gm, dict(group_list=fake(I64, 5)), B.ERR_SHAPE),
    (gm, dict(y=fake(BF, 299, 384)), B.ERR_SHAPE),
    (gm, dict(activation=1), B.ERR_SHAPE),
    (gm, dict(n=24, activation=1, y=fake(BF, 300, 12)), B.ERR_SHAPE),
    (mx, dict(k=544), B.ERR_SHAPE),
    (mx, dict(x_scale=fake(E8, 300, 16)), B.ERR_SHAPE),
    (mx, dict(w_scale=fake(E8, 4, 384, 9, 2)), B.ERR_SHAPE),
    (gm, dict(m=2 ** 31, y=fake(BF, 2 ** 31, 384)), B.ERR_SHAPE),
    (gm, dict(k=65536, n=65536, transpose_w=1, activation=1, w=fake(BF, 4, 65536, 65536), y=fake(BF, 300, 32768)),
     B.ERR_SHAPE),
    (gm, dict(x=fake(BF, 300, 512, ptr=0x7000008)), B.ERR_ALIGN),
    (mx, dict(w_scale=fake(E8, 4, 384, 8, 2, ptr=0x7000002)), B.ERR_ALIGN),
]


@pytest.mark.parametrize("make,over,code", GM_CASES, ids=[str(i) for i in range(len(GM_CASES))])
def test_product_stage_one(make, over, code):
    sizes = {k: v for k, v in over.items() if k in ("m", "k", "n", "e", "dt", "xt")}
    a = make(**sizes, **{k: v for k, v in over.items() if k not in sizes})
    st, ws = stage_one("gmm_grouped_matmul", a)
    assert st == code
    if code != B.OK:
        assert ws == 12345
        assert B.lib().gmm_grouped_matmul(ctypes.byref(a), None, 0, None) == code  # before any launch


GW_CASES = [
    ({}, B.OK), (dict(dt=F16), B.OK), (dict(dw=fake(BF, 4, 512, 384)), B.OK), (dict(accumulate=1), B.OK),
    (dict(m=0), B.OK), (dict(tuning=[0, 128]), B.OK),
    (dict(dy=B.Tensor()), B.ERR_NULLPTR),
    (dict(dw=B.Tensor()), B.ERR_NULLPTR),
    (dict(dt=F32), B.ERR_DTYPE),
    (dict(dy=fake(F16, 300, 384)), B.ERR_DTYPE),
    (dict(dw=fake(F16, 4, 512, 384)), B.ERR_DTYPE),
    (dict(group_list=fake(F32, 4)), B.ERR_DTYPE),
    (dict(accumulate=2), B.ERR_ATTR),
    (dict(accumulate=1, dw=fake(BF, 4, 512, 384)), B.ERR_ATTR),
    (dict(group_list_type=-1), B.ERR_ATTR),
    (dict(tuning=[0, 32]), B.ERR_ATTR),
    (dict(k=12), B.ERR_SHAPE), (dict(n=12), B.ERR_SHAPE),
    (dict(dy=fake(BF, 301, 384)), B.ERR_SHAPE),
    (dict(dw=fake(F32, 4, 384, 512)), B.ERR_SHAPE),
    (dict(dw=fake(F32, 4, 512, 384, ptr=0x7000004)), B.ERR_ALIGN),
]


@pytest.mark.parametrize("over,code", GW_CASES, ids=[str(i) for i in range(len(GW_CASES))])
def test_wgrad_stage_one(over, code):
    sizes = {k: v for k, v in over.items() if k in ("m", "k", "n", "e", "dt")}
    a = gw(**sizes, **{k: v for k, v in over.items() if k not in sizes})
    st, ws = stage_one("gmm_grouped_matmul_wgrad", a)
    assert st == code
    if code != B.OK:
        assert ws == 12345
        assert B.lib().gmm_grouped_matmul_wgrad(ctypes.byref(a), None, 0, None) == code


def mq(x, codes, scales, transpose=0):
    a = B.MqArgs()
    a.x, a.codes, a.scales, a.transpose = x, codes, scales, transpose
    return a


MQ_CASES = [
    (mq(B.Tensor(), fake(FP4, 8, 32), fake(E8, 8, 1, 2)), B.ERR_NULLPTR),
    (mq(fake(BF, 8, 64), B.Tensor(), fake(E8, 8, 1, 2)), B.ERR_NULLPTR),
    (mq(fake(B.DT_INT8, 8, 64), fake(FP4, 8, 32), fake(E8, 8, 1, 2)), B.ERR_DTYPE),
    (mq(fake(BF, 8, 64), fake(B.DT_INT8, 8, 32), fake(E8, 8, 1, 2)), B.ERR_DTYPE),
    (mq(fake(BF, 8, 64), fake(FP4, 8, 32), fake(F32, 8, 1, 2)), B.ERR_DTYPE),
    (mq(fake(BF, 2, 64, 8), fake(FP4, 2, 8, 32), fake(E8, 2, 8, 1, 2), 2), B.ERR_ATTR),
    (mq(fake(BF, 64, 8), fake(FP4, 8, 32), fake(E8, 8, 1, 2), 1), B.ERR_SHAPE),
    (mq(fake(BF, 8, 96), fake(FP4, 8, 48), fake(E8, 8, 1, 2)), B.ERR_SHAPE),
    (mq(fake(BF, 8, 64), fake(FP4, 8, 64), fake(E8, 8, 1, 2)), B.ERR_SHAPE),
    (mq(fake(BF, 8, 64), fake(FP8, 8, 32), fake(E8, 8, 1, 2)), B.ERR_SHAPE),
    (mq(fake(BF, 8, 64), fake(FP4, 8, 32), fake(E8, 8, 2)), B.ERR_SHAPE),
    (mq(fake(BF, 2, 64, 12), fake(FP4, 2, 12, 32), fake(E8, 2, 12, 1, 2), 1), B.ERR_SHAPE),
    (mq(fake(BF, 3, 8, 64), fake(FP4, 2, 8, 32), fake(E8, 3, 8, 1, 2)), B.ERR_SHAPE),
    (mq(fake(BF, 8, 64, ptr=0x7000002), fake(FP4, 8, 32), fake(E8, 8, 1, 2)), B.ERR_ALIGN),
]


@pytest.mark.parametrize("a,code", MQ_CASES, ids=[str(i) for i in range(len(MQ_CASES))])
def test_quantise_rejects(a, code):
    assert B.lib().gmm_mx_quantize(ctypes.byref(a), None) == code
    assert B.lib().gmm_mx_dequantize(ctypes.byref(a), None) == (B.ERR_ATTR if a.transpose else code)


def test_packed_descriptors_are_the_structs():
    """The binding fills a call's structs in one go: field by field the same as _desc's."""
    x, w = torch.zeros((8, 64), dtype=torch.bfloat16), torch.zeros((2, 64, 16), dtype=torch.bfloat16)
    gl, y = torch.tensor([4, 8]), torch.zeros((8, 16), dtype=torch.bfloat16)
    a, keep = B.make_gm_args(x, w, gl, y, group_list_type=1, transpose_w=False, activation="swiglu", tuning_config=[5, 32])
    for name, t in (("x", x), ("w", w), ("group_list", gl), ("y", y), ("x_scale", None)):
        d, want = getattr(a, name), B._desc(t)
        assert (d.data, d.dtype, d.ndim, list(d.dims)[:d.ndim]) == (want.data, want.dtype, want.ndim, list(want.dims)[:want.ndim])
    assert (a.group_list_type, a.transpose_w, a.activation, a.tuning_config_len) == (1, 0, 1, 2)
    assert list(a.tuning_config[:2]) == [5, 32]
    g, _ = B.make_gw_args(x, y, gl, torch.zeros((2, 64, 16)), accumulate=True)
    assert (g.accumulate, g.group_list_type, g.dw.dtype, bool(g.tuning_config)) == (1, 0, B.DT_FLOAT32, False)


def test_python_entry_refuses_host_tensors():
    """A pointer of another device would be dereferenced by the kernels."""
    x, w = torch.zeros((8, 64), dtype=torch.bfloat16), torch.zeros((2, 64, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.grouped_matmul(x, w, torch.tensor([4, 8]))
    with pytest.raises(ValueError):
        B.grouped_matmul_wgrad(x, x, torch.tensor([4, 8]))
    with pytest.raises(ValueError):
        B.mx_quantize(x)
    with pytest.raises(ValueError):
        B.mx_dequantize(x, x)


def test_python_entry_refuses_strided_tensors():
    x = torch.zeros((64, 8), dtype=torch.bfloat16).T
    with pytest.raises(ValueError):
        B.make_mq_args(x, x, x)


def qp(x1, pts, k=2048, T=512, K=8):
    a = B.QpArgs()
    a.hidden, a.expert_ids, a.row_index, a.group_list = fake(BF, T, k), fake(I64, T, K), fake(I64, T * K), fake(I64, 32)
    a.x1, a.pertoken_scale, a.group_list_type = x1, pts, 1
    return a


@pytest.mark.parametrize("a,code", [
    (qp(fake(FP4, 4096, 1024), fake(E8, 4096, 32, 2)), B.OK),
    (qp(fake(FP4, 4096, 1024), fake(F32, 4096)), B.ERR_DTYPE),
    (qp(fake(FP4, 4096, 2048), fake(E8, 4096, 32, 2)), B.ERR_SHAPE),
    (qp(fake(FP4, 4096, 1024), fake(E8, 4096, 64)), B.ERR_SHAPE),
    (qp(fake(FP4, 4096, 1040), fake(E8, 4096, 32, 2), k=2080), B.ERR_SHAPE),
], ids=["ok", "scale_dtype", "codes_unpacked", "scale_shape", "k_not_mult_64"])
def test_producer_step_with_fp4_rows(a, code):
    st, _ = stage_one("gmm_quant_permute", a)
    assert st == code
