"""The gated block of a layer as a torch.autograd.Function, to be taken as it
stands, under gradients of every layout that autograd hands to it."""
import numpy as np
import pytest
import torch
from torch.autograd.function import once_differentiable

from quantized_moe_grouped_amd import binding as B

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


class GatedBlock(torch.autograd.Function):
    """y = (act(x w1[..., :f]) * (x w1[..., f:])) w2 for rows of x grouped by
    expert (counts), kept in FP8 for w1's gradient; w1 (e,k,2f), w2 (e,f,d).
    keep: "full" or "fp8", of the projections.  Rows behind the last group have
    no part: those of y and of x's gradient are whatever their memory held."""

    @staticmethod
    def forward(ctx, x, w1, w2, counts, act="swiglu", keep="fp8"):
        h, kept, scale = B.gated_matmul(x, w1, counts, activation=act, keep=keep, group_list_type=1)
        codes, x_scale = B.mx_quantize(x, format="fp8")
        ctx.save_for_backward(codes, x_scale, kept, scale, w1, w2, counts)
        ctx.act = act
        return B.grouped_matmul(h, w2, counts, group_list_type=1)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        codes, x_scale, kept, scale, w1, w2, counts = ctx.saved_tensors
        dy = dy.contiguous()  # behind a sum it is expanded, behind a transpose turned
        d, h = B.gated_matmul_backward(dy, w2, counts, kept, kept_scale=scale, activation=ctx.act, group_list_type=1)
        dx = B.grouped_matmul(d, w1, counts, transpose_w=True, group_list_type=1)
        dw1 = B.grouped_matmul_wgrad(codes, d, counts, x_scale=x_scale, out_dtype=w1.dtype, group_list_type=1)
        dw2 = B.grouped_matmul_wgrad(h, dy, counts, out_dtype=w2.dtype, group_list_type=1)
        return dx, dw1, dw2, None, None, None


def _leaves(seed=3):
    rng = np.random.default_rng(seed)
    shapes = (((70, 128), 1.0), ((3, 128, 192), 0.1), ((3, 96, 128), 0.1))
    return [(torch.from_numpy(rng.standard_normal(s)) * scale).to(BF16).cuda().requires_grad_() for s, scale in shapes]


COUNTS = [30, 0, 40]
LOSSES = {  # of y, and what backward is handed: none of these is contiguous
    "sum": lambda y: y.sum(),
    "mean of rows": lambda y: y.float().mean(0).square().sum(),
    "turned": lambda y: (y.T.contiguous() * torch.arange(70, device="cuda")).sum(),
    "half of the columns": lambda y: y[:, ::2].float().square().sum(),
}


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("keep", ["full", "fp8"])
@pytest.mark.parametrize("loss", LOSSES)
def test_gradients_of_every_layout(loss, keep, act):
    """To the bit those of the same gradient laid out."""
    leaves, counts = _leaves(), torch.tensor(COUNTS).cuda()
    y = GatedBlock.apply(*leaves, counts, act, keep)
    got = torch.autograd.grad(LOSSES[loss](y), leaves, retain_graph=True)
    alone = y.detach().requires_grad_()
    dy, = torch.autograd.grad(LOSSES[loss](alone), alone)
    want = torch.autograd.grad(y, leaves, dy.contiguous())
    for g, w, leaf in zip(got, want, leaves):
        assert g.shape == leaf.shape and g.dtype == leaf.dtype
        assert torch.equal(g, w) and torch.isfinite(g).all() and g.abs().sum() > 0


def test_it_learns_nothing_from_other_rows():
    """Rows behind the last group, and an expert without rows, have no part."""
    leaves, counts = _leaves(), torch.tensor([30, 0, 30]).cuda()
    y = GatedBlock.apply(*leaves, counts)
    dx, dw1, dw2 = torch.autograd.grad(y[:60].sum(), leaves)
    assert (dw1[1] == 0).all() and (dw2[1] == 0).all()
    x = leaves[0].detach()[:60].requires_grad_()
    short = GatedBlock.apply(x, *leaves[1:], counts)
    assert torch.equal(short, y[:60])
    for a, b in zip(torch.autograd.grad(short.sum(), [x, *leaves[1:]]), (dx[:60], dw1, dw2)):
        assert torch.equal(a, b)


def test_a_second_derivative_is_refused():
    leaves, counts = _leaves(), torch.tensor(COUNTS).cuda()
    dx, = torch.autograd.grad(GatedBlock.apply(*leaves, counts).float().square().sum(), leaves[:1], create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()
