"""What a call returns is its own launch's status: an error that the program
made earlier, and has not asked for yet, is neither reported nor taken away."""
import ctypes

import pytest
import torch

from quantized_moe_grouped_amd import binding as B

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture
def earlier_error():
    """Leaves an error of an invalid host argument (no device work) in the
    runtime's last-error slot; gives the runtime's way to read and clear it."""
    hip = ctypes.CDLL("libamdhip64.so.7")

    def make():
        torch.cuda.synchronize()
        hip.hipGetLastError()
        status = hip.hipSetDevice(9999)
        assert status != 0
        return status
    yield make, hip.hipGetLastError
    hip.hipGetLastError()


def test_an_earlier_error_is_not_the_calls_own(earlier_error):
    make, last = earlier_error
    x = torch.ones((40, 64), dtype=BF16, device="cuda")
    w = torch.ones((2, 64, 32), dtype=BF16, device="cuda")
    gl = torch.tensor([10, 40], device="cuda")
    y, dw = torch.empty((40, 32), dtype=BF16, device="cuda"), torch.empty((2, 64, 32), device="cuda")
    codes, scales = B.mx_quantize(x)
    values = torch.empty_like(x)
    gm, keep1 = B.make_gm_args(x, w, gl, y)
    gw, keep2 = B.make_gw_args(x, y, gl, dw)
    mq, keep3 = B.make_mq_args(x, codes, scales)
    md, keep4 = B.make_mq_args(values, codes, scales)
    L, stream = B.lib(), torch.cuda.current_stream().cuda_stream
    calls = [lambda: L.gmm_grouped_matmul(ctypes.byref(gm), None, 0, stream),
             lambda: L.gmm_grouped_matmul_wgrad(ctypes.byref(gw), None, 0, stream),
             lambda: L.gmm_mx_quantize(ctypes.byref(mq), stream),
             lambda: L.gmm_mx_dequantize(ctypes.byref(md), stream)]
    for i, call in enumerate(calls):
        status = make()
        got, left = call(), last()
        assert got == B.OK, i
        assert left == status, i
    torch.cuda.synchronize()
    assert (y == 64).all() and torch.equal(values, x)
