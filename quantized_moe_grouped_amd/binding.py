"""ctypes binding of libgmmfr.so -- argument marshalling only.

Every step of the computation runs in the HIP library; this module turns torch
tensors into the C descriptors of include/gmmfr.h and forwards the current HIP
stream.  It raises when the library is missing: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgmmfr.so")

# status codes (gmmfr_status)
OK, ERR_NULLPTR, ERR_DTYPE, ERR_SHAPE, ERR_ATTR, ERR_UNSUPPORTED, ERR_ALIGN, ERR_WORKSPACE, ERR_HIP = range(9)
STATUS_NAMES = {0: "OK", 1: "NULLPTR", 2: "DTYPE", 3: "SHAPE", 4: "ATTR", 5: "UNSUPPORTED", 6: "ALIGN",
                7: "WORKSPACE", 8: "HIP"}
# element types (gmmfr_dtype)
DT_NONE, DT_INT8, DT_INT4, DT_INT32, DT_INT64, DT_FLOAT32, DT_BFLOAT16 = range(7)
DT_FLOAT8_E4M3FN, DT_FLOAT4_E2M1X2, DT_FLOAT8_E8M0, DT_FLOAT16 = 7, 8, 9, 10
COMBINE = {"auto": 0, "atomic": 1, "ordered": 2}
COMBINE_HYBRID = 3  # reported by the plan only

EXPORTED = ("gmm_finalize_routing_workspace", "gmm_finalize_routing", "gmm_finalize_routing_profiled",
            "gmm_finalize_routing_plan", "gmmfr_status_string", "gmm_quant_permute_workspace",
            "gmm_quant_permute", "gmm_quant_permute_profiled", "gmm_finalize_routing_noalloc",
            "gmm_grouped_matmul_workspace", "gmm_grouped_matmul", "gmm_grouped_matmul_wgrad_workspace",
            "gmm_grouped_matmul_wgrad", "gmm_mx_quantize", "gmm_mx_dequantize", "gmm_grouped_matmul_plan",
            "gmm_gated_matmul_workspace", "gmm_gated_matmul", "gmm_gated_matmul_backward_workspace",
            "gmm_gated_matmul_backward", "gmm_grouped_matmul_wgrad_fp8_workspace", "gmm_grouped_matmul_wgrad_fp8",
            "gmm_grouped_matmul_wgrad_plan", "gmm_grouped_matmul_wgrad_fp8_plan", "gmm_gated_matmul_plan",
            "gmm_gated_matmul_backward_plan")
ACTIVATION = {None: 0, "none": 0, "swiglu": 1}
GATE = {"swiglu": 1, "geglu": 2}  # of the gated block
NOALLOC_SCRATCH_BYTES = 128 << 20  # GMMFR_NOALLOC_SCRATCH_BYTES


class GmmfrError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        self.status = STATUS_NAMES.get(code, str(code))
        super().__init__(f"{where}: {self.status}")


class Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("dims", ctypes.c_int64 * 4)]


class Args(ctypes.Structure):
    _fields_ = [
        ("x1", Tensor), ("x2", Tensor), ("scale", Tensor),
        ("bias", Tensor), ("offset", Tensor), ("antiquant_scale", Tensor), ("antiquant_offset", Tensor),
        ("pertoken_scale", Tensor), ("group_list", Tensor), ("shared_input", Tensor), ("logit", Tensor),
        ("row_index", Tensor), ("out", Tensor), ("acc_out", Tensor),
        ("group_list_type", ctypes.c_int64), ("shared_input_offset", ctypes.c_int64), ("output_bs", ctypes.c_int64),
        ("transpose_x1", ctypes.c_int32), ("transpose_x2", ctypes.c_int32),
        ("deterministic", ctypes.c_int32), ("combine", ctypes.c_int32),
        ("tuning_config", ctypes.POINTER(ctypes.c_int64)), ("tuning_config_len", ctypes.c_int64),
    ]


class QpArgs(ctypes.Structure):
    _fields_ = [
        ("hidden", Tensor), ("expert_ids", Tensor), ("topk_weights", Tensor), ("x1", Tensor),
        ("pertoken_scale", Tensor), ("logit", Tensor), ("row_index", Tensor), ("group_list", Tensor),
        ("expert_offset", ctypes.c_int64), ("group_list_type", ctypes.c_int64),
    ]


class GmArgs(ctypes.Structure):
    _fields_ = [
        ("x", Tensor), ("w", Tensor), ("x_scale", Tensor), ("w_scale", Tensor), ("group_list", Tensor), ("y", Tensor),
        ("group_list_type", ctypes.c_int64), ("transpose_w", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("tuning_config", ctypes.POINTER(ctypes.c_int64)), ("tuning_config_len", ctypes.c_int64),
    ]


class GmPlanInfo(ctypes.Structure):
    _fields_ = [("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("grid", ctypes.c_int32)]


class GwArgs(ctypes.Structure):
    _fields_ = [
        ("x", Tensor), ("dy", Tensor), ("group_list", Tensor), ("dw", Tensor),
        ("group_list_type", ctypes.c_int64), ("accumulate", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("tuning_config", ctypes.POINTER(ctypes.c_int64)), ("tuning_config_len", ctypes.c_int64),
    ]


class GxArgs(ctypes.Structure):
    _fields_ = [
        ("x", Tensor), ("dy", Tensor), ("x_scale", Tensor), ("dy_scale", Tensor), ("group_list", Tensor), ("dw", Tensor),
        ("group_list_type", ctypes.c_int64), ("accumulate", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("tuning_config", ctypes.POINTER(ctypes.c_int64)), ("tuning_config_len", ctypes.c_int64),
    ]


class GfArgs(ctypes.Structure):
    _fields_ = [
        ("x", Tensor), ("w", Tensor), ("group_list", Tensor), ("h", Tensor), ("kept", Tensor), ("kept_scale", Tensor),
        ("group_list_type", ctypes.c_int64), ("transpose_w", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("tuning_config", ctypes.POINTER(ctypes.c_int64)), ("tuning_config_len", ctypes.c_int64),
    ]


class GbArgs(ctypes.Structure):
    _fields_ = [
        ("dy", Tensor), ("w", Tensor), ("group_list", Tensor), ("kept", Tensor), ("kept_scale", Tensor), ("d", Tensor),
        ("h", Tensor), ("group_list_type", ctypes.c_int64), ("transpose_w", ctypes.c_int32),
        ("activation", ctypes.c_int32), ("tuning_config", ctypes.POINTER(ctypes.c_int64)),
        ("tuning_config_len", ctypes.c_int64),
    ]


_PLANS = {GmArgs: "gmm_grouped_matmul_plan", GwArgs: "gmm_grouped_matmul_wgrad_plan", GxArgs: "gmm_grouped_matmul_wgrad_fp8_plan",
          GfArgs: "gmm_gated_matmul_plan", GbArgs: "gmm_gated_matmul_backward_plan"}


class MqArgs(ctypes.Structure):
    _fields_ = [("x", Tensor), ("codes", Tensor), ("scales", Tensor), ("transpose", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("combine", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("tile_k", ctypes.c_int32), ("grid", ctypes.c_int32), ("int4_weights", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_int64), ("gemm_kernel", ctypes.c_char * 96),
                ("hybrid_atomic", ctypes.c_int32)]


_lib = None


def lib():
    """The loaded library; raises when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m quantized_moe_grouped_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.gmm_finalize_routing_workspace.argtypes = [ctypes.POINTER(Args), ctypes.POINTER(ctypes.c_size_t)]
        L.gmm_finalize_routing_workspace.restype = ctypes.c_int
        L.gmm_finalize_routing.argtypes = [ctypes.POINTER(Args), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        L.gmm_finalize_routing.restype = ctypes.c_int
        L.gmm_finalize_routing_profiled.argtypes = [ctypes.POINTER(Args), ctypes.c_void_p, ctypes.c_size_t,
                                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
        L.gmm_finalize_routing_profiled.restype = ctypes.c_int
        L.gmm_finalize_routing_noalloc.argtypes = [ctypes.POINTER(Args), ctypes.c_void_p]
        L.gmm_finalize_routing_noalloc.restype = ctypes.c_int
        L.gmm_finalize_routing_plan.argtypes = [ctypes.POINTER(Args), ctypes.POINTER(PlanInfo)]
        L.gmm_finalize_routing_plan.restype = ctypes.c_int
        L.gmm_quant_permute_workspace.argtypes = [ctypes.POINTER(QpArgs), ctypes.POINTER(ctypes.c_size_t)]
        L.gmm_quant_permute_workspace.restype = ctypes.c_int
        L.gmm_quant_permute.argtypes = [ctypes.POINTER(QpArgs), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        L.gmm_quant_permute.restype = ctypes.c_int
        L.gmm_quant_permute_profiled.argtypes = [ctypes.POINTER(QpArgs), ctypes.c_void_p, ctypes.c_size_t,
                                                 ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
        L.gmm_quant_permute_profiled.restype = ctypes.c_int
        # arguments of these as void*: a struct by reference, or its bytes
        for name in ("gmm_grouped_matmul", "gmm_grouped_matmul_wgrad", "gmm_grouped_matmul_wgrad_fp8", "gmm_gated_matmul",
                     "gmm_gated_matmul_backward"):
            getattr(L, name + "_workspace").argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)]
            getattr(L, name + "_workspace").restype = ctypes.c_int
            getattr(L, name).argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name + "_plan").argtypes = [ctypes.c_void_p, ctypes.POINTER(GmPlanInfo)]
            getattr(L, name + "_plan").restype = ctypes.c_int
        for name in ("gmm_mx_quantize", "gmm_mx_dequantize"):
            getattr(L, name).argtypes = [ctypes.c_void_p, ctypes.c_void_p]
            getattr(L, name).restype = ctypes.c_int
        L.gmmfr_status_string.argtypes = [ctypes.c_int]
        L.gmmfr_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _dtype_code(t, int4_packed: bool = False) -> int:
    import torch
    if t.dtype == torch.int8:
        return DT_INT8
    if t.dtype == torch.int32:
        return DT_INT32
    if t.dtype == torch.int64:
        return DT_INT64
    if t.dtype == torch.float32:
        return DT_FLOAT32
    if t.dtype == torch.bfloat16:
        return DT_BFLOAT16
    if t.dtype == torch.float8_e4m3fn:
        return DT_FLOAT8_E4M3FN
    if t.dtype == torch.float4_e2m1fn_x2:
        return DT_FLOAT4_E2M1X2
    if t.dtype == torch.float8_e8m0fnu:
        return DT_FLOAT8_E8M0
    raise TypeError(f"unsupported tensor dtype {t.dtype}")


def _desc(t, dtype: Optional[int] = None) -> Tensor:
    d = Tensor()
    if t is None:
        return d
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if t.dim() > 4:
        raise ValueError("at most 4 dimensions")
    d.data = t.data_ptr()
    d.dtype = _dtype_code(t) if dtype is None else dtype
    d.ndim = t.dim()
    for i, s in enumerate(t.shape):
        d.dims[i] = int(s)
    return d


def make_args(x1, x2, group_list, out, *, scale=None, pertoken_scale=None, logit=None, row_index=None,
              shared_input=None, shared_input_offset: int = 0, group_list_type: int = 0,
              deterministic: bool = False, combine: str = "auto", acc_out=None,
              tuning_config: Optional[Sequence[int]] = None, bias=None, offset=None,
              antiquant_scale=None, antiquant_offset=None, transpose_x1: bool = False,
              transpose_x2: bool = False):
    """Build the C argument struct.  Returns (args, keepalive): the struct holds
    raw device pointers, so keep `keepalive` (which references every tensor
    passed, and the host tuning array) alive until the call has been enqueued
    and the stream has reached it."""
    a = Args()
    a.x1 = _desc(x1)
    a.x2 = _desc(x2)
    a.scale = _desc(scale)
    a.bias = _desc(bias)
    a.offset = _desc(offset)
    a.antiquant_scale = _desc(antiquant_scale)
    a.antiquant_offset = _desc(antiquant_offset)
    a.pertoken_scale = _desc(pertoken_scale)
    a.group_list = _desc(group_list)
    a.shared_input = _desc(shared_input)
    a.logit = _desc(logit)
    a.row_index = _desc(row_index)
    a.out = _desc(out)
    a.acc_out = _desc(acc_out)
    a.group_list_type = int(group_list_type)
    a.shared_input_offset = int(shared_input_offset)
    a.output_bs = int(out.shape[0]) if out is not None else 0
    a.transpose_x1 = int(bool(transpose_x1))
    a.transpose_x2 = int(bool(transpose_x2))
    a.deterministic = int(bool(deterministic))
    a.combine = COMBINE[combine]
    tuning = None
    if tuning_config:
        tuning = (ctypes.c_int64 * len(tuning_config))(*[int(v) for v in tuning_config])
        a.tuning_config = ctypes.cast(tuning, ctypes.POINTER(ctypes.c_int64))
        a.tuning_config_len = len(tuning_config)
    keep = (x1, x2, group_list, out, scale, pertoken_scale, logit, row_index, shared_input, acc_out, bias, offset,
            antiquant_scale, antiquant_offset, tuning)
    return a, keep


def workspace_size(args: Args) -> int:
    n = ctypes.c_size_t(0)
    st = lib().gmm_finalize_routing_workspace(ctypes.byref(args), ctypes.byref(n))
    if st != OK:
        raise GmmfrError(st, "gmm_finalize_routing_workspace")
    return int(n.value)


def plan(args: Args) -> dict:
    info = PlanInfo()
    st = lib().gmm_finalize_routing_plan(ctypes.byref(args), ctypes.byref(info))
    if st != OK:
        raise GmmfrError(st, "gmm_finalize_routing_plan")
    return {"combine": {1: "atomic", 2: "ordered", 3: "hybrid"}[info.combine], "tile_m": info.tile_m,
            "tile_n": info.tile_n, "tile_k": info.tile_k, "grid": info.grid, "int4_weights": bool(info.int4_weights),
            "workspace_bytes": int(info.workspace_bytes), "gemm_kernel": info.gemm_kernel.decode(),
            "hybrid_atomic": int(info.hybrid_atomic)}


def _torch_stream(stream):
    """The torch stream object for `stream`: None (the current stream), a
    torch.cuda.Stream, or a raw hipStream_t handle."""
    import torch
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream
    if int(stream) == 0:  # the null stream
        return torch.cuda.default_stream()
    return torch.cuda.ExternalStream(int(stream))


def run(args: Args, workspace=None, stream=None) -> None:
    """Enqueue on `stream` (default: torch's current stream on the current device)."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    ws_ptr = 0 if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().gmm_finalize_routing(ctypes.byref(args), ctypes.c_void_p(ws_ptr), ctypes.c_size_t(ws_bytes),
                                    ctypes.c_void_p(stream))
    if st != OK:
        raise GmmfrError(st, "gmm_finalize_routing")


def gmm_finalize_routing(x1, x2, group_list, out, *, workspace=None, stream=None, **kw) -> None:
    """One call: validate, size the workspace, allocate it with torch if none
    is given, enqueue.  Keyword arguments are those of make_args.

    A workspace allocated here is taken from the pool of the stream the kernels
    run on, so when it is released on return the caching allocator hands the
    block out again only to work ordered after them on that stream (a block
    from another stream's pool could be reused, and overwritten, while the
    kernels still run)."""
    import torch
    args, keep = make_args(x1, x2, group_list, out, **kw)
    need = workspace_size(args)
    ts = _torch_stream(stream)
    if need and workspace is None:
        with torch.cuda.stream(ts):
            workspace = torch.empty(need, dtype=torch.uint8, device=out.device)
    run(args, workspace, ts)
    del keep


def run_noalloc(args: Args, stream=None) -> None:
    """Enqueue through the allocation-free entry point (the library's own
    scratch array; nothing is allocated) on `stream` (default: the current
    stream)."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    st = lib().gmm_finalize_routing_noalloc(ctypes.byref(args), ctypes.c_void_p(stream))
    if st != OK:
        raise GmmfrError(st, "gmm_finalize_routing_noalloc")


def gmm_finalize_routing_noalloc(x1, x2, group_list, out, *, stream=None, **kw) -> None:
    """gmm_finalize_routing without any allocation (see run_noalloc).
    Keyword arguments are those of make_args."""
    args, keep = make_args(x1, x2, group_list, out, **kw)
    run_noalloc(args, stream)
    del keep


# ---------------------------------------------------------------- producer step


def make_qp_args(hidden, expert_ids, x1, pertoken_scale, row_index, group_list, *, topk_weights=None,
                 logit=None, expert_offset: int = 0, group_list_type: int = 1):
    """C arguments of gmm_quant_permute.  hidden is bf16 (T,k) and expert_ids
    int32/int64 (T,K); the outputs are x1 int8 (T*K,k), pertoken_scale fp32
    (T*K), row_index int32/int64 (T*K), group_list int64 (e), and logit fp32
    (T*K) when topk_weights (T,K) is given.  Returns (args, keepalive)."""
    a = QpArgs()
    a.hidden = _desc(hidden)
    a.expert_ids = _desc(expert_ids)
    a.topk_weights = _desc(topk_weights)
    a.x1 = _desc(x1)
    a.pertoken_scale = _desc(pertoken_scale)
    a.logit = _desc(logit)
    a.row_index = _desc(row_index)
    a.group_list = _desc(group_list)
    a.expert_offset = int(expert_offset)
    a.group_list_type = int(group_list_type)
    return a, (hidden, expert_ids, topk_weights, x1, pertoken_scale, logit, row_index, group_list)


def qp_workspace_size(args: QpArgs) -> int:
    n = ctypes.c_size_t(0)
    st = lib().gmm_quant_permute_workspace(ctypes.byref(args), ctypes.byref(n))
    if st != OK:
        raise GmmfrError(st, "gmm_quant_permute_workspace")
    return int(n.value)


def quant_permute(hidden, expert_ids, num_experts: int, *, topk_weights=None, expert_offset: int = 0,
                  group_list_type: int = 1, row_index_dtype=None, mode: str = "int8", workspace=None,
                  stream=None) -> dict:
    """Allocate the outputs with torch and enqueue gmm_quant_permute on `stream`
    (default: the current stream).  mode: "int8" (int8 x1, fp32 per-token
    scale), "fp8" (FP8 E4M3 x1, fp32 per-token scale), "mx" (FP8 E4M3 x1,
    E8M0 scale per 32 values, (m, k/64, 2)) or "mx4" (FP4 E2M1 x1 (m, k/2),
    scales as "mx").  Returns the output tensors by name."""
    import torch
    dev = hidden.device
    T, k = hidden.shape
    K = expert_ids.shape[1]
    m = T * K
    ts = _torch_stream(stream)
    with torch.cuda.stream(ts):  # outputs and workspace from the pool of the stream that writes them
        return _quant_permute_on(hidden, expert_ids, num_experts, topk_weights, expert_offset, group_list_type,
                                 row_index_dtype, mode, workspace, ts, dev, T, k, m)


def _quant_permute_on(hidden, expert_ids, num_experts, topk_weights, expert_offset, group_list_type,
                      row_index_dtype, mode, workspace, ts, dev, T, k, m):
    import torch
    if mode == "int8":
        x1 = torch.empty((m, k), dtype=torch.int8, device=dev)
        pts = torch.empty(m, dtype=torch.float32, device=dev)
    elif mode == "fp8":
        x1 = torch.empty((m, k), dtype=torch.float8_e4m3fn, device=dev)
        pts = torch.empty(m, dtype=torch.float32, device=dev)
    elif mode == "mx":
        x1 = torch.empty((m, k), dtype=torch.float8_e4m3fn, device=dev)
        pts = torch.empty((m, k // 64, 2), dtype=torch.float8_e8m0fnu, device=dev)
    elif mode == "mx4":
        x1 = torch.empty((m, k // 2), dtype=torch.float4_e2m1fn_x2, device=dev)
        pts = torch.empty((m, k // 64, 2), dtype=torch.float8_e8m0fnu, device=dev)
    else:
        raise ValueError(f"unknown mode {mode!r}")
    out = dict(x1=x1,
               pertoken_scale=pts,
               row_index=torch.empty(m, dtype=row_index_dtype or torch.int64, device=dev),
               group_list=torch.empty(num_experts, dtype=torch.int64, device=dev),
               logit=None if topk_weights is None else torch.empty(m, dtype=torch.float32, device=dev))
    args, keep = make_qp_args(hidden, expert_ids, out["x1"], out["pertoken_scale"], out["row_index"],
                              out["group_list"], topk_weights=topk_weights, logit=out["logit"],
                              expert_offset=expert_offset, group_list_type=group_list_type)
    need = qp_workspace_size(args)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    stream = ts.cuda_stream
    ws_ptr = 0 if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().gmm_quant_permute(ctypes.byref(args), ctypes.c_void_p(ws_ptr), ctypes.c_size_t(ws_bytes),
                                 ctypes.c_void_p(stream))
    if st != OK:
        raise GmmfrError(st, "gmm_quant_permute")
    del keep
    out["workspace"] = workspace
    return out


# ------------------------------------------------- grouped products and MX quantisation

_pack_tensor = struct.Struct("=Qii4q").pack
_pack_qii = struct.Struct("=qii").pack
_pack_ii = struct.Struct("=ii").pack
_ABSENT = _pack_tensor(0, 0, 0, 0, 0, 0, 0)
_PAD = {n: (0,) * (4 - n) for n in range(5)}
_codes_of: dict = {}


def _packed(t) -> bytes:
    """The bytes of a gmmfr_tensor (these calls are short: one struct, filled
    at once, instead of a field at a time)."""
    if t is None:
        return _ABSENT
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    shape = t.shape
    if len(shape) > 4:
        raise ValueError("at most 4 dimensions")
    code = _codes_of.get(t.dtype)
    if code is None:
        import torch
        code = DT_FLOAT16 if t.dtype == torch.float16 else _dtype_code(t)
        _codes_of[t.dtype] = code
    return _pack_tensor(t.data_ptr(), code, len(shape), *shape, *_PAD[len(shape)])


def _packed_tuning(tuning_config):
    """(host array or None, the two fields' bytes)"""
    if not tuning_config:
        return None, bytes(16)
    tuning = (ctypes.c_int64 * len(tuning_config))(*[int(v) for v in tuning_config])
    return tuning, struct.pack("=Qq", ctypes.addressof(tuning), len(tuning_config))


def _gm_bytes(x, w, group_list, y, x_scale, w_scale, group_list_type, transpose_w, activation, tail) -> bytes:
    return b"".join((_packed(x), _packed(w), _packed(x_scale), _packed(w_scale), _packed(group_list), _packed(y),
                     _pack_qii(group_list_type, bool(transpose_w), ACTIVATION[activation]), tail))


def _gw_bytes(x, dy, group_list, dw, group_list_type, accumulate, tail) -> bytes:
    return b"".join((_packed(x), _packed(dy), _packed(group_list), _packed(dw),
                     _pack_qii(group_list_type, bool(accumulate), 0), tail))


def _mq_bytes(x, codes, scales, transpose) -> bytes:
    return b"".join((_packed(x), _packed(codes), _packed(scales), _pack_ii(bool(transpose), 0)))


def _gx_bytes(x, dy, x_scale, dy_scale, group_list, dw, group_list_type, accumulate, tail) -> bytes:
    return b"".join((_packed(x), _packed(dy), _packed(x_scale), _packed(dy_scale), _packed(group_list), _packed(dw),
                     _pack_qii(group_list_type, bool(accumulate), 0), tail))


def _gf_bytes(x, w, group_list, h, kept, kept_scale, group_list_type, transpose_w, activation, tail) -> bytes:
    return b"".join((_packed(x), _packed(w), _packed(group_list), _packed(h), _packed(kept), _packed(kept_scale),
                     _pack_qii(group_list_type, bool(transpose_w), GATE[activation]), tail))


def _gb_bytes(dy, w, group_list, kept, kept_scale, d, h, group_list_type, transpose_w, activation, tail) -> bytes:
    return b"".join((_packed(dy), _packed(w), _packed(group_list), _packed(kept), _packed(kept_scale), _packed(d),
                     _packed(h), _pack_qii(group_list_type, bool(transpose_w), GATE[activation]), tail))


def make_gm_args(x, w, group_list, y, *, x_scale=None, w_scale=None, group_list_type: int = 0,
                 transpose_w: bool = False, activation: Optional[str] = None,
                 tuning_config: Optional[Sequence[int]] = None):
    """C arguments of gmm_grouped_matmul.  Returns (args, keepalive), as make_args."""
    tuning, tail = _packed_tuning(tuning_config)
    raw = _gm_bytes(x, w, group_list, y, x_scale, w_scale, group_list_type, transpose_w, activation, tail)
    return GmArgs.from_buffer_copy(raw), (x, w, group_list, y, x_scale, w_scale, tuning)


def gm_plan(args) -> dict:
    """The plan that gmm_grouped_matmul, gmm_grouped_matmul_wgrad(_fp8),
    gmm_gated_matmul or gmm_gated_matmul_backward takes, by the struct that the
    arguments are (host only)."""
    name = _PLANS[type(args)]
    info = GmPlanInfo()
    st = getattr(lib(), name)(ctypes.byref(args), ctypes.byref(info))
    if st != OK:
        raise GmmfrError(st, name)
    return {"tile_m": info.tile_m, "tile_n": info.tile_n, "grid": info.grid}


def make_gw_args(x, dy, group_list, dw, *, group_list_type: int = 0, accumulate: bool = False,
                 tuning_config: Optional[Sequence[int]] = None):
    """C arguments of gmm_grouped_matmul_wgrad.  Returns (args, keepalive)."""
    tuning, tail = _packed_tuning(tuning_config)
    raw = _gw_bytes(x, dy, group_list, dw, group_list_type, accumulate, tail)
    return GwArgs.from_buffer_copy(raw), (x, dy, group_list, dw, tuning)


def make_gx_args(x, dy, group_list, dw, *, x_scale=None, dy_scale=None, group_list_type: int = 0,
                 accumulate: bool = False, tuning_config: Optional[Sequence[int]] = None):
    """C arguments of gmm_grouped_matmul_wgrad_fp8.  Returns (args, keepalive)."""
    tuning, tail = _packed_tuning(tuning_config)
    raw = _gx_bytes(x, dy, x_scale, dy_scale, group_list, dw, group_list_type, accumulate, tail)
    return GxArgs.from_buffer_copy(raw), (x, dy, x_scale, dy_scale, group_list, dw, tuning)


def make_gf_args(x, w, group_list, h, *, kept=None, kept_scale=None, group_list_type: int = 0,
                 transpose_w: bool = False, activation: str = "swiglu", tuning_config: Optional[Sequence[int]] = None):
    """C arguments of gmm_gated_matmul.  Returns (args, keepalive)."""
    tuning, tail = _packed_tuning(tuning_config)
    raw = _gf_bytes(x, w, group_list, h, kept, kept_scale, group_list_type, transpose_w, activation, tail)
    return GfArgs.from_buffer_copy(raw), (x, w, group_list, h, kept, kept_scale, tuning)


def make_gb_args(dy, w, group_list, kept, d, *, kept_scale=None, h=None, group_list_type: int = 0,
                 transpose_w: bool = True, activation: str = "swiglu", tuning_config: Optional[Sequence[int]] = None):
    """C arguments of gmm_gated_matmul_backward.  Returns (args, keepalive)."""
    tuning, tail = _packed_tuning(tuning_config)
    raw = _gb_bytes(dy, w, group_list, kept, kept_scale, d, h, group_list_type, transpose_w, activation, tail)
    return GbArgs.from_buffer_copy(raw), (dy, w, group_list, kept, kept_scale, d, h, tuning)


def make_mq_args(x, codes, scales, *, transpose: bool = False):
    """C arguments of gmm_mx_quantize and gmm_mx_dequantize.  Returns (args, keepalive)."""
    return MqArgs.from_buffer_copy(_mq_bytes(x, codes, scales, transpose)), (x, codes, scales)


def _check_tensors(x, *others):
    """The device of x.  No tensor may want a gradient that these calls would
    lose (they record no history), nor carry a tangent of forward-mode
    differentiation (they read the values alone), and all live on one GPU,
    where the kernels dereference their pointers."""
    import torch
    dev, wanting, elsewhere = x.device, x.requires_grad, None
    for t in others:
        if t is not None:
            wanting = wanting or t.requires_grad
            if t.device != dev:
                elsewhere = t.device
    if wanting and torch.is_grad_enabled():
        raise ValueError("these calls record no gradients: detach the tensors, or call them under torch.no_grad() or "
                         "in a torch.autograd.Function of your own")
    dual = torch.autograd.forward_ad
    if dual._current_level >= 0:  # (none outside of a dual level; looked up for each tensor it would cost 2 us a call)
        for t in (x, *others):
            if t is not None and dual.unpack_dual(t).tangent is not None:
                raise ValueError("these calls carry no tangents of forward-mode differentiation: unpack the tensors, or "
                                 "call them in a torch.autograd.Function with a jvp of your own")
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, not on {dev}")
    if elsewhere is not None:
        raise ValueError(f"tensors must be on one device: {elsewhere} and {dev}")
    return dev


def _on(dev, stream, call, *args):
    """call(raw stream handle, *args) with `dev` current and, where a stream is
    given, that stream too (so that what the call allocates comes from its pool).
    Tensors among args are then marked as used on it: freed on return, their
    memory waits for the kernels before it is handed out again.  (Not on a
    stream that the caller made outside torch, and may destroy: there the
    caller keeps them alive.)"""
    import torch
    if stream is None and torch.cuda.current_device() == dev.index:
        return call(torch._C._cuda_getCurrentRawStream(dev.index), *args)
    with torch.cuda.device(dev):
        ts = _torch_stream(stream)
        if ts.device != dev:
            raise ValueError(f"the stream is on {ts.device}, the tensors on {dev}")
        with torch.cuda.stream(ts):
            result = call(ts.cuda_stream, *args)
        if not isinstance(ts, torch.cuda.ExternalStream):
            for t in args:
                if isinstance(t, torch.Tensor):
                    t.record_stream(ts)
        return result


def _enqueue(name: str, raw: bytes, workspace, handle) -> None:
    """Stage 2.  These calls want no workspace (stage 1 says 0 bytes), but for the
    weight gradient of FP8 rows, sometimes; one that is given is passed on."""
    ptr, size = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = getattr(lib(), name)(raw, ptr, size, handle)
    if st != OK:
        raise GmmfrError(st, name)


def grouped_matmul(x, w, group_list, *, x_scale=None, w_scale=None, out=None, out_dtype=None,
                   group_list_type: int = 0, transpose_w: bool = False, activation: Optional[str] = None,
                   tuning_config: Optional[Sequence[int]] = None, workspace=None, stream=None):
    """Rows of x, sorted by expert and split by group_list, times their
    expert's weights; activation "swiglu": silu of the product's first n/2
    columns times the others.  16-bit x and w (weights (e,k,n), or (e,n,k) with
    transpose_w: then this is also the gradient towards the rows of a product
    with (e,k,n) weights), or microscaled x (FP8 or FP4) and FP4 w (e,n,k) with
    their scales.  Returns out, allocated as (m, n or n/2) if none is given, in
    out_dtype (default: x's type; bf16 for microscaled x); rows behind the last
    group are left as they are.  Records no history: tensors that want a
    gradient are refused (see also grouped_matmul_wgrad)."""
    dev = _check_tensors(x, w, group_list, x_scale, w_scale, out, workspace)
    return _on(dev, stream, _grouped_matmul, x, w, group_list, x_scale, w_scale, out, out_dtype, group_list_type,
               transpose_w, activation, tuning_config, workspace)


def _grouped_matmul(handle, x, w, group_list, x_scale, w_scale, out, out_dtype, group_list_type, transpose_w,
                    activation, tuning_config, workspace):
    import torch
    if out is None:
        columns = w.shape[1 if transpose_w else 2] // (2 if ACTIVATION[activation] else 1)
        dtype = out_dtype or (x.dtype if x.dtype in (torch.bfloat16, torch.float16) else torch.bfloat16)
        out = torch.empty((x.shape[0], columns), dtype=dtype, device=x.device)
    tuning, tail = _packed_tuning(tuning_config)
    raw = _gm_bytes(x, w, group_list, out, x_scale, w_scale, group_list_type, transpose_w, activation, tail)
    _enqueue("gmm_grouped_matmul", raw, workspace, handle)
    del tuning  # the host array lives until the call has read it
    return out


def grouped_matmul_wgrad(x, dy, group_list, *, x_scale=None, dy_scale=None, out=None, out_dtype=None,
                         accumulate: bool = False, group_list_type: int = 0,
                         tuning_config: Optional[Sequence[int]] = None, workspace=None, stream=None):
    """Gradient of a grouped product's weights (e,k,n): x_g^T dy_g for every
    expert, in out_dtype (default fp32), zeros for one without rows.
    accumulate: added to `out` (fp32).  Weights kept as (e,n,k): pass (dy, x).
    One of the two may be in FP8 with its scales (x_scale or dy_scale, as
    mx_quantize makes them): the result is that of the same values in the other
    operand's type (beside an fp16 operand those past 65504 are infinite, and
    those below 2^-14 lose bits), but for the order of additions where the rows
    of few, long groups are split (a workspace is allocated then, if none is
    given).  With a gate dy is the gradient of the product before it
    (gated_matmul_backward)."""
    dev = _check_tensors(x, dy, group_list, x_scale, dy_scale, out, workspace)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    return _on(dev, stream, _grouped_matmul_wgrad, x, dy, group_list, x_scale, dy_scale, out, out_dtype, accumulate,
               group_list_type, tuning_config, workspace)


def _grouped_matmul_wgrad(handle, x, dy, group_list, x_scale, dy_scale, out, out_dtype, accumulate, group_list_type,
                          tuning_config, workspace):
    import torch
    if out is None:
        out = torch.empty((group_list.shape[0], x.shape[1], dy.shape[1]), dtype=out_dtype or torch.float32,
                          device=x.device)
    tuning, tail = _packed_tuning(tuning_config)
    if x_scale is None and dy_scale is None:
        raw = _gw_bytes(x, dy, group_list, out, group_list_type, accumulate, tail)
        _enqueue("gmm_grouped_matmul_wgrad", raw, workspace, handle)
    else:
        raw = _gx_bytes(x, dy, x_scale, dy_scale, group_list, out, group_list_type, accumulate, tail)
        try:
            _enqueue("gmm_grouped_matmul_wgrad_fp8", raw, workspace, handle)
        except GmmfrError as e:
            if workspace is not None or e.code != ERR_WORKSPACE:
                raise
            need = ctypes.c_size_t(0)  # one is wanted: nothing was launched without it
            lib().gmm_grouped_matmul_wgrad_fp8_workspace(raw, ctypes.byref(need))
            workspace = torch.empty(need.value, dtype=torch.uint8, device=x.device)
            _enqueue("gmm_grouped_matmul_wgrad_fp8", raw, workspace, handle)
    del tuning
    return out


def _check_gate(activation):
    if activation not in GATE:
        raise ValueError(f"unknown activation {activation!r}: one of {', '.join(GATE)}")


def gated_matmul(x, w, group_list, *, activation: str = "swiglu", keep: Optional[str] = None, out=None, kept=None,
                 kept_scale=None, group_list_type: int = 0, transpose_w: bool = False,
                 tuning_config: Optional[Sequence[int]] = None, workspace=None, stream=None):
    """The gated feed-forward block of every expert (or, with one group, of a
    dense layer): act(x w[..., :f]) * (x w[..., f:]), act silu ("swiglu") or
    gelu in its tanh form ("geglu").  16-bit x (m,k) and w (e,k,2f), or (e,2f,k)
    with transpose_w.  keep: the two projections for gated_matmul_backward, in
    x's type ("full") or in FP8 with one scale per 32 columns ("fp8", as
    mx_quantize makes them; f % 32 == 0), or not (None).  Returns (h, kept,
    kept_scale): h (m,f) in x's type, kept (m,2f), kept_scale (m,2f/64,2), the
    last two None where there are none; `out`, `kept` and `kept_scale` are
    written to where they are given.  Rows behind the last group are left as
    they are.  Records no history: tensors that want a gradient are refused."""
    _check_gate(activation)
    if keep not in (None, "full", "fp8"):
        raise ValueError(f"unknown keep {keep!r}: None, 'full' or 'fp8'")
    if (kept is not None and keep is None) or (kept_scale is not None and keep != "fp8"):
        raise ValueError("a buffer for what is kept needs keep to say so")
    dev = _check_tensors(x, w, group_list, out, kept, kept_scale, workspace)
    return _on(dev, stream, _gated_matmul, x, w, group_list, activation, keep, out, kept, kept_scale, group_list_type,
               transpose_w, tuning_config, workspace)


def _gated_matmul(handle, x, w, group_list, activation, keep, out, kept, kept_scale, group_list_type, transpose_w,
                  tuning_config, workspace):
    import torch
    m, both = x.shape[0], w.shape[1 if transpose_w else 2]
    if out is None:
        out = torch.empty((m, both // 2), dtype=x.dtype, device=x.device)
    if keep is not None and kept is None:
        kept = torch.empty((m, both), dtype=x.dtype if keep == "full" else torch.float8_e4m3fn, device=x.device)
    if keep == "fp8" and kept_scale is None:
        kept_scale = torch.empty((m, both // 64, 2), dtype=torch.float8_e8m0fnu, device=x.device)
    tuning, tail = _packed_tuning(tuning_config)
    raw = _gf_bytes(x, w, group_list, out, kept, kept_scale, group_list_type, transpose_w, activation, tail)
    _enqueue("gmm_gated_matmul", raw, workspace, handle)
    del tuning
    return out, kept, kept_scale


def gated_matmul_backward(dy, w, group_list, kept, *, kept_scale=None, activation: str = "swiglu", out=None, h=None,
                          want_h: bool = True, group_list_type: int = 0, transpose_w: bool = True,
                          tuning_config: Optional[Sequence[int]] = None, workspace=None, stream=None):
    """The way back through gated_matmul, from dy (m,d), the gradient behind the
    block's last projection with weights w (e,f,d), or (e,d,f) with transpose_w
    = False: dh = dy w^T through the gate to the gradients of the two
    projections, side by side as (m,2f), and h = act(u) v again (m,f), from what
    gated_matmul kept.  Returns (d, h), h None without want_h; written to `out`
    and `h` where they are given.  The other gradients, with w1 the projections'
    weights (e,k,2f) and x the block's rows:
    grouped_matmul(d, w1, ..., transpose_w=True) for x,
    grouped_matmul_wgrad(x, d, ...) for w1, grouped_matmul_wgrad(h, dy, ...) for
    w.  Rows behind the last group are left as they are.  Records no history."""
    _check_gate(activation)
    if h is not None and not want_h:
        raise ValueError("h is given but not wanted")
    dev = _check_tensors(dy, w, group_list, kept, kept_scale, out, h, workspace)
    return _on(dev, stream, _gated_matmul_backward, dy, w, group_list, kept, kept_scale, activation, out, h, want_h,
               group_list_type, transpose_w, tuning_config, workspace)


def _gated_matmul_backward(handle, dy, w, group_list, kept, kept_scale, activation, out, h, want_h, group_list_type,
                           transpose_w, tuning_config, workspace):
    import torch
    m, f = dy.shape[0], w.shape[1 if transpose_w else 2]
    if out is None:
        out = torch.empty((m, 2 * f), dtype=dy.dtype, device=dy.device)
    if want_h and h is None:
        h = torch.empty((m, f), dtype=dy.dtype, device=dy.device)
    tuning, tail = _packed_tuning(tuning_config)
    raw = _gb_bytes(dy, w, group_list, kept, kept_scale, out, h, group_list_type, transpose_w, activation, tail)
    _enqueue("gmm_gated_matmul_backward", raw, workspace, handle)
    del tuning
    return out, h


def mx_quantize(x, *, format: str = "fp4", transpose: bool = False, stream=None):
    """(codes, scales) of x (rows,k) or (e,n,k), or with transpose of weights
    (e,k,n), which become (e,n,k): FP4 (k/2 bytes a row) or FP8 codes with one
    E8M0 scale per 32 values, (..., k/64, 2)."""
    if format not in ("fp4", "fp8"):
        raise ValueError(f"unknown format {format!r}")
    if transpose and x.dim() != 3:
        raise ValueError("transpose takes weights (e,k,n)")
    return _on(_check_tensors(x), stream, _mx_quantize, x, format, transpose)


def _mx_quantize(handle, x, format, transpose):
    import torch
    shape = x.shape
    lead, k = ((shape[0], shape[2]), shape[1]) if transpose else (shape[:-1], shape[-1])
    if format == "fp4":
        codes = torch.empty((*lead, k // 2), dtype=torch.float4_e2m1fn_x2, device=x.device)
    else:
        codes = torch.empty((*lead, k), dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty((*lead, k // 64, 2), dtype=torch.float8_e8m0fnu, device=x.device)
    st = lib().gmm_mx_quantize(_mq_bytes(x, codes, scales, transpose), handle)
    if st != OK:
        raise GmmfrError(st, "gmm_mx_quantize")
    return codes, scales


def mx_dequantize(codes, scales, *, dtype=None, stream=None):
    """The values that codes and scales stand for, (rows,k) or (e,n,k), in
    dtype (bf16 by default, fp16 or fp32)."""
    return _on(_check_tensors(codes, scales), stream, _mx_dequantize, codes, scales, dtype)


def _mx_dequantize(handle, codes, scales, dtype):
    import torch
    shape = codes.shape
    per = 2 if codes.dtype == torch.float4_e2m1fn_x2 else 1
    x = torch.empty((*shape[:-1], shape[-1] * per), dtype=dtype or torch.bfloat16, device=codes.device)
    st = lib().gmm_mx_dequantize(_mq_bytes(x, codes, scales, False), handle)
    if st != OK:
        raise GmmfrError(st, "gmm_mx_dequantize")
    return x
