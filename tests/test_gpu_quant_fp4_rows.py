"""The producer step's FP4 rows, bit for bit: codes and scales of the tokens by
grouped_ref.encode, the routing by the oracle's permute.  Hidden sizes for each
of the kernel's forms: rows held in registers (up to 2048 and 4096 values) and
rows read twice (longer)."""
import numpy as np
import pytest
import torch

from oracle import quant as Q
from quantized_moe_grouped_amd import binding as B
from quantized_moe_grouped_amd import workloads as W
from tests import grouped_ref as R

pytestmark = pytest.mark.gpu


def _check(rp, row_index_dtype=torch.int64):
    hidden = torch.from_numpy(rp.hidden.view(np.int16)).cuda().view(torch.bfloat16)
    weights = None if rp.topk_weights is None else torch.from_numpy(rp.topk_weights).cuda()
    got = B.quant_permute(hidden, torch.from_numpy(np.ascontiguousarray(rp.expert_ids)).cuda(), rp.e, topk_weights=weights,
                          expert_offset=rp.expert_offset, group_list_type=rp.group_list_type,
                          row_index_dtype=row_index_dtype, mode="mx4")
    order, counts = Q.permute(rp.expert_ids, rp.e, rp.expert_offset)
    rows, token = len(order), order // rp.K
    if rows:
        codes, scales = R.pack(*R.encode(Q.bf16_to_f32(rp.hidden), "fp4"), "fp4")
        assert torch.equal(got["x1"].view(torch.uint8).cpu()[:rows], codes.view(torch.uint8)[token])
        assert torch.equal(got["pertoken_scale"].view(torch.uint8).cpu()[:rows], scales.view(torch.uint8)[token])
    assert np.array_equal(got["row_index"].cpu().numpy()[:rows], token)
    assert np.array_equal(got["group_list"].cpu().numpy(), np.cumsum(counts) if rp.group_list_type == 0 else counts)
    if weights is None:
        assert got["logit"] is None
    else:
        assert np.array_equal(got["logit"].cpu().numpy()[:rows], rp.topk_weights.reshape(-1)[order])


@pytest.mark.parametrize("k", [64, 1984, 2048, 2112, 4096, 4160, 7168, 8256])
@pytest.mark.parametrize("tokens,top,experts", [(1, 1, 1), (90, 2, 4), (333, 8, 16)])
def test_fp4_rows(k, tokens, top, experts):
    _check(W.route_problem(k + tokens, tokens, k, top, experts))


@pytest.mark.parametrize("kw", [
    dict(T=300, k=256, K=8, e=16, n_gate=64, expert_offset=16, ids_dtype=np.int32, group_list_type=0),
    dict(T=257, k=4096, K=3, e=5, zero_tokens=4, repeat_slots=True),
    dict(T=257, k=7168, K=3, e=5, zero_tokens=4, repeat_slots=True),
    dict(T=0, k=64, K=2, e=4),
    dict(T=200, k=2112, K=8, e=1024),
], ids=["offset", "zeros_4096", "zeros_7168", "no_tokens", "experts_1024"])
def test_fp4_rows_of_other_routings(kw):
    _check(W.route_problem(seed=41, **kw), torch.int32)


def test_fp4_rows_without_weights():
    rp = W.route_problem(42, 50, 4160, 2, 3)
    rp.topk_weights = None
    _check(rp)


def test_fp4_rows_over_the_exponents():
    """Blocks from bf16's subnormal values to its largest."""
    rng = np.random.default_rng(43)
    for k in (320, 2240, 7168):
        rp = W.route_problem(44, 60, k, 2, 3)
        rp.hidden = rng.integers(0, 0x7F80, rp.hidden.shape).astype(np.uint16) | (
            rng.integers(0, 2, rp.hidden.shape) << 15).astype(np.uint16)
        small = rng.random((60, k // 32)) < 0.5  # half of the blocks below 2^-100, some of them all subnormal
        top = rng.choice([0x0001, 0x007F, 0x0100, 0x0D00], (60, k // 32))
        blocks = rp.hidden.reshape(60, -1, 32)
        blocks[small] = (blocks[small] & 0x8000) | ((blocks[small] & 0x7FFF) % (top[small] + 1)[:, None])
        _check(rp)


@pytest.mark.parametrize("seed", range(20))
def test_drawn_fp4_rows(seed):
    rng = np.random.default_rng(31000 + seed)
    tokens, top = int(rng.choice([1, 33, 500, 2000])), int(rng.integers(1, 9))
    experts, offset = int(rng.choice([4, 32, 300, 1024])), int(rng.choice([0, 0, 8]))
    n_gate = experts + offset + int(rng.choice([0, 5]))
    rp = W.route_problem(31000 + seed, tokens, 64 * int(rng.integers(1, 130)), min(top, n_gate), experts, n_gate=n_gate,
                         expert_offset=offset, ids_dtype=np.int32 if rng.random() < 0.4 else np.int64,
                         with_weights=bool(rng.random() < 0.8), group_list_type=int(rng.integers(2)),
                         zero_tokens=int(rng.integers(0, 3)), repeat_slots=bool(rng.random() < 0.2))
    _check(rp, torch.int32 if rng.random() < 0.3 else torch.int64)


def test_fp4_rows_of_the_dispatch_workload():
    """16384 tokens, k = 2048, top-8 of 32 experts, against the whole oracle."""
    rp = W.make_route_config("dispatch", 0)
    rp.mode = "mx4"
    ref = Q.run(rp)
    hidden = torch.from_numpy(rp.hidden.view(np.int16)).cuda().view(torch.bfloat16)
    got = B.quant_permute(hidden, torch.from_numpy(rp.expert_ids).cuda(), rp.e,
                          topk_weights=torch.from_numpy(rp.topk_weights).cuda(), group_list_type=rp.group_list_type, mode="mx4")
    rows = ref["rows"]
    assert np.array_equal(got["x1"].view(torch.uint8).cpu().numpy()[:rows], ref["x1"][:rows])
    assert np.array_equal(got["pertoken_scale"].view(torch.uint8).cpu().numpy().reshape(len(ref["x1"]), -1)[:rows],
                          ref["pertoken_scale"][:rows])
    assert np.array_equal(got["row_index"].cpu().numpy()[:rows], ref["row_index"][:rows])
    assert np.array_equal(got["group_list"].cpu().numpy(), ref["group_list"])
    assert np.array_equal(got["logit"].cpu().numpy()[:rows], ref["logit"][:rows])
