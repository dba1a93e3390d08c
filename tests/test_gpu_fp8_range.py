"""FP8 with block scales over the whole range of both: what the gated block keeps,
and what the weight gradient makes of kept rows."""
import numpy as np
import pytest
import torch

from quantized_moe_grouped_amd import binding as B
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("side", ["x", "dy"])
@pytest.mark.parametrize("height", [128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_every_code_under_every_scale(dtype, height, side):
    """A row is a group of its own and the other operand one, so that results are
    single values: the nearest of the type (infinity past its range, subnormals
    kept), NaN for the NaN codes and the NaN scale."""
    m, k = 256, 8192
    codes = torch.arange(256, dtype=torch.uint8).repeat(32).expand(m, k).contiguous().view(torch.float8_e4m3fn)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].expand(m, k // 32).reshape(m, k // 64, 2).contiguous().view(torch.float8_e8m0fnu)
    want = R.decode(codes, scales).to(dtype).float()
    other = torch.zeros((m, 8), dtype=dtype, device="cuda")
    other[:, 3] = 1
    c, s, gl = codes.cuda(), scales.cuda(), torch.ones(m, dtype=torch.int64).cuda()
    kw = dict(group_list_type=1, tuning_config=[0, height])
    if side == "x":
        got = B.grouped_matmul_wgrad(c, other, gl, x_scale=s, **kw)[:, :, 3]
    else:
        got = B.grouped_matmul_wgrad(other, c, gl, dy_scale=s, **kw)[:, 3]
    got = got.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[~got.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("height", [32, 128, 256])
def test_blocks_of_every_size_are_kept_as_mx_quantisation_keeps_them(height):
    """One row of x picks one row of w, so that the sums are the weights: blocks
    from the subnormals to the largest bf16 numbers, and of zeros."""
    rng = np.random.default_rng(4)
    m, f = 8, 4096
    size = np.arange(2 * f // 32).reshape(-1, 1) - 133.0  # of each block: 2^-133 .. 2^122
    both = rng.uniform(-1, 1, (m, 2 * f // 32, 32)) * 2.0 ** size * 2.0 ** rng.integers(0, 5, (m, 1, 1))
    both[:, ::17] = 0
    both = torch.from_numpy(both.reshape(m, 2 * f)).to(BF16)
    x, w = torch.eye(m, dtype=BF16), both[None].contiguous()
    _, kept, scale = B.gated_matmul(x.cuda(), w.cuda(), torch.tensor([m]).cuda(), keep="fp8", tuning_config=[0, height])
    codes, want = R.pack(*R.encode(both.float().numpy(), "fp8"), "fp8")
    assert torch.equal(scale.cpu().view(torch.uint8), want.view(torch.uint8))
    got, codes = kept.cpu().view(torch.uint8), codes.view(torch.uint8)
    assert torch.equal(got & 127, codes & 127)
    assert torch.equal(got[(got & 127) != 0], codes[(got & 127) != 0])  # (a sum of zero has no sign to speak of)
    q, s = B.mx_quantize(both.float().cuda(), format="fp8")
    assert torch.equal(s.cpu().view(torch.uint8), want.view(torch.uint8)) and torch.equal(q.cpu().view(torch.uint8) & 127, got & 127)
