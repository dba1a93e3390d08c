"""A tensor with a tangent of forward-mode differentiation does not want a
gradient, and the kernels would read its values alone: such a call is refused
before anything else is looked at (no GPU needed)."""
import pytest
import torch
from torch.autograd import forward_ad

from quantized_moe_grouped_amd import binding as B

BF16, FP8, E8 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu


def _tensors():
    return dict(x=torch.zeros((8, 64), dtype=BF16), w=torch.zeros((2, 64, 64), dtype=BF16), dy=torch.zeros((8, 16), dtype=BF16),
                w2=torch.zeros((2, 32, 16), dtype=BF16), kept=torch.zeros((8, 64), dtype=BF16), out=torch.zeros((2, 64, 16)))


def _calls(x, w, dy, w2, kept, out):
    gl = torch.tensor([4, 8])
    codes, scales = torch.zeros((8, 64), dtype=torch.uint8).view(FP8), torch.zeros((8, 1, 2), dtype=torch.uint8).view(E8)
    return {
        "product": lambda: B.grouped_matmul(x, w, gl),
        "wgrad": lambda: B.grouped_matmul_wgrad(x, dy, gl, out=out, accumulate=True),
        "wgrad of FP8 rows": lambda: B.grouped_matmul_wgrad(codes, dy, gl, x_scale=scales, out=out),
        "gated": lambda: B.gated_matmul(x, w, gl),
        "gated, back": lambda: B.gated_matmul_backward(dy, w2, gl, kept),
        "quantize": lambda: B.mx_quantize(x),
    }


CALLS = [("product", "x"), ("product", "w"), ("wgrad", "x"), ("wgrad", "dy"), ("wgrad", "out"), ("wgrad of FP8 rows", "dy"),
         ("wgrad of FP8 rows", "out"), ("gated", "x"), ("gated", "w"), ("gated, back", "dy"), ("gated, back", "w2"),
         ("gated, back", "kept"), ("quantize", "x")]


@pytest.mark.parametrize("call,which", CALLS)
def test_a_lost_tangent_is_refused(call, which):
    t = _tensors()
    with forward_ad.dual_level():
        t[which] = forward_ad.make_dual(t[which], torch.ones_like(t[which]))
        assert not t[which].requires_grad
        with pytest.raises(ValueError, match="tangent"):
            _calls(**t)[call]()
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):  # which leaves forward mode on
            _calls(**t)[call]()
        t[which] = forward_ad.unpack_dual(t[which]).primal
        with pytest.raises(ValueError, match="GPU"):  # the next check answers
            _calls(**t)[call]()
    with pytest.raises(ValueError, match="GPU"):
        _calls(**_tensors())[call]()


def test_functional_transforms_are_refused_too():
    t = _tensors()
    with pytest.raises(ValueError, match="tangent"):
        torch.func.jvp(lambda x: _calls(**{**t, "x": x})["gated"](), (t["x"],), (t["x"],))


def test_a_function_with_its_own_jvp_may_call_them():
    """Inside its forward the tangents are its own affair."""
    t = _tensors()

    class Own(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            with pytest.raises(ValueError, match="GPU"):
                _calls(**{**t, "x": x})["gated"]()
            return x * 2

        @staticmethod
        def jvp(ctx, dx):
            return dx * 2

    with forward_ad.dual_level():
        y = forward_ad.unpack_dual(Own.apply(forward_ad.make_dual(t["x"], torch.ones_like(t["x"]))))
        assert (y.tangent == 2).all()
