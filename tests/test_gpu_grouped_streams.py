"""Tensors handed to a call on another stream than their own and freed on
return: their memory is not given to new tensors before the kernels are done."""
import pytest
import torch

from quantized_moe_grouped_amd import binding as B

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _calls():
    """Calls on inputs of their own (1 MiB or more each: blocks of their own), and what they give."""
    gl = torch.tensor([512, 1024], device="cuda")
    x = torch.randn((1024, 1024), device="cuda").to(BF16)
    w = torch.randn((2, 1024, 512), device="cuda").to(BF16)
    dy = torch.randn((1024, 512), device="cuda").to(BF16)
    codes, scales = B.mx_quantize(x, format="fp8")
    return {
        "product": (lambda s, x, w: B.grouped_matmul(x, w, gl, stream=s), (x, w)),
        "wgrad": (lambda s, x, dy: B.grouped_matmul_wgrad(x, dy, gl, stream=s), (x, dy)),
        "quantize": (lambda s, x: B.mx_quantize(x, format="fp8", stream=s), (x,)),
        "dequantize": (lambda s, c, sc: B.mx_dequantize(c, sc, stream=s), (codes, scales)),
    }


def _bytes(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("name", ["product", "wgrad", "quantize", "dequantize"])
def test_inputs_freed_before_the_side_stream_comes_to_them(name):
    call, inputs = _calls()[name]
    want = call(None, *inputs)
    want = want if isinstance(want, tuple) else (want,)
    side = torch.cuda.Stream()
    temporary = [torch.empty_like(t) for t in inputs]
    for t, v in zip(temporary, inputs):
        t.copy_(v)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms in front of the call
    got = call(side, *temporary)
    shapes = [(t.shape, t.dtype) for t in temporary]
    del temporary, t
    # what takes a freed block's place is written on the current stream at once
    new = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(3)]
    for t in new:
        _bytes(t).fill_(0x7F)
    torch.cuda.synchronize()
    for g, w in zip(got if isinstance(got, tuple) else (got,), want):
        assert torch.equal(_bytes(g), _bytes(w)), name
    del new


def test_in_a_captured_graph():
    """A call with a stream of its own inside a capture, joined to it, replayed
    with new inputs and eager work between."""
    call, (x, w) = _calls()["product"]
    side = torch.cuda.Stream()
    call(None, x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        y = call(side, x, w)
        torch.cuda.current_stream().wait_stream(side)
    for step in range(3):
        x.copy_(torch.randn(x.shape, device="cuda"))
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, call(None, x, w)), step


def test_a_stream_of_the_callers_own():
    """A raw handle: nothing is left with the allocator that needs it later."""
    call, (x, w) = _calls()["product"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = call(side.cuda_stream, x, w)
    side.synchronize()
    assert torch.equal(y, call(None, x, w))
