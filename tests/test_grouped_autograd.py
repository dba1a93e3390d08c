"""The grouped products and the MX quantisation record no history for automatic
differentiation: a call that would lose a gradient is refused, with what to
write instead, before anything else is looked at (no GPU needed)."""
import pytest
import torch

from quantized_moe_grouped_amd import binding as B

BF16 = torch.bfloat16


def _calls(x, w, dy, out=None):
    gl = torch.tensor([4, 8])
    codes = torch.zeros((8, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros((8, 1, 2), dtype=torch.uint8).view(torch.float8_e8m0fnu)
    return {
        "product": lambda: B.grouped_matmul(x, w, gl, out=out),
        "wgrad": lambda: B.grouped_matmul_wgrad(x, dy, gl),
        "quantize": lambda: B.mx_quantize(x),
        "dequantize": lambda: B.mx_dequantize(codes, scales),
    }


def _tensors():
    return dict(x=torch.zeros((8, 64), dtype=BF16), w=torch.zeros((2, 64, 16), dtype=BF16),
                dy=torch.zeros((8, 16), dtype=BF16), out=torch.zeros((8, 16), dtype=BF16))


@pytest.mark.parametrize("call,which", [("product", "x"), ("product", "w"), ("product", "out"), ("wgrad", "x"),
                                        ("wgrad", "dy"), ("quantize", "x")])
def test_a_lost_gradient_is_refused(call, which):
    t = _tensors()
    t[which].requires_grad_()
    with pytest.raises(ValueError, match="no_grad"):
        _calls(**t)[call]()


@pytest.mark.parametrize("call", ["product", "wgrad", "quantize"])
def test_without_gradients_they_are_taken(call):
    """Under no_grad, or detached, the next check is the one that answers."""
    t = _tensors()
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        _calls(**{k: v.requires_grad_() for k, v in t.items()})[call]()
    with pytest.raises(ValueError, match="GPU"):
        _calls(**{k: v.detach() for k, v in t.items()})[call]()
    with pytest.raises(ValueError, match="GPU"):
        _calls(**_tensors())["dequantize"]()
