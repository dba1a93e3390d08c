"""The producer oracle's FP4 rows against the table-driven encoding of the MX
formats, which shares no code with it."""
import numpy as np
import pytest

from oracle import quant as Q
from quantized_moe_grouped_amd import workloads as W
from tests import grouped_ref as R


def _same(bits):
    got, scale = Q.quantize_mx4(bits)
    code, want = R.encode(Q.bf16_to_f32(bits), "fp4")
    assert np.array_equal(scale, want)
    assert np.array_equal(got, code[:, 0::2] | code[:, 1::2] << 4)


def test_every_finite_bf16_value():
    """Each as the largest of its block beside smaller ones, of both signs."""
    top = np.arange(0x7F80, dtype=np.uint16)
    rng = np.random.default_rng(1)
    x = (rng.random((len(top), 32)) * (top[:, None].astype(np.int64) + 1)).astype(np.uint16)
    x[:, 7] = top
    _same(x | (rng.integers(0, 2, x.shape) << 15).astype(np.uint16))


@pytest.mark.parametrize("scale", [2.0 ** -100, 1.0, 2.0 ** 100])
def test_ties(scale):
    v = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7], dtype=np.float32)
    x = np.concatenate([v, -v]) * np.float32(scale)
    _same((x.view(np.uint32) >> 16).astype(np.uint16)[None])


def test_a_whole_problem():
    rp = W.route_problem(3, 70, 192, 3, 5)
    rp.mode = "mx4"
    r = Q.run(rp)
    assert r["x1"].shape == (210, 96) and r["pertoken_scale"].shape == (210, 6)
    codes, scales = Q.quantize_mx4(rp.hidden)
    assert np.array_equal(r["x1"][:r["rows"]], codes[r["row_index"][:r["rows"]]])
    assert np.array_equal(r["pertoken_scale"][:r["rows"]], scales[r["row_index"][:r["rows"]]])


def test_what_is_refused():
    with pytest.raises(ValueError):
        Q.quantize_mx4(np.zeros((2, 48), dtype=np.uint16))
    with pytest.raises(ValueError):
        Q.quantize_mx4(np.full((1, 32), 0x7F80, dtype=np.uint16))
