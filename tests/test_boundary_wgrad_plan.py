"""Which tile the weight gradient takes for few rows an expert, on both sides of
each bound (host only, fake pointers)."""
import pytest

from quantized_moe_grouped_amd import binding as B
from tests.test_boundary_gated import gx
from tests.test_boundary_grouped import BF, F16, fake, gw


def _tile(e, k, n, rows, out=BF, **over):
    return B.gm_plan(gw(m=e * rows, k=k, n=n, e=e, dw=fake(out, e, k, n), **over))["tile_m"]


@pytest.mark.parametrize("e,k,n,rows,tile", [
    # 256-row tiles of two rounds at most (512 of them), and of more
    (4, 2048, 2048, 8, 128), (8, 2048, 2048, 64, 128), (12, 2048, 2048, 64, 256), (4, 4096, 2048, 64, 128),
    (4, 4096, 4096, 64, 256),
    # a sixteenth less work for the smaller: the ends of rounds, and of matrices
    (4, 7168, 2048, 64, 128), (16, 7168, 2048, 64, 256), (64, 2880, 2880, 64, 128), (64, 1408, 2048, 64, 128),
    (16, 5120, 1536, 64, 128), (64, 5120, 1536, 64, 256),
    # a row for each 512 columns of k, from 2048 on
    (16, 4096, 8192, 8, 128), (16, 4096, 8192, 9, 256), (64, 2048, 2048, 4, 128), (64, 2048, 2048, 5, 256),
    (64, 1024, 4096, 1, 256), (64, 1024, 1024, 64, 256), (16, 2048, 4096, 16, 256),
    # more rows: by the rounds alone
    (4, 2048, 2048, 64, 128), (4, 2048, 2048, 65, 256), (64, 2880, 2880, 65, 256),
])
def test_results_of_16_bits(e, k, n, rows, tile):
    assert _tile(e, k, n, rows) == tile


@pytest.mark.parametrize("e,k,n,rows", [(4, 2048, 2048, 8), (64, 2880, 2880, 8), (16, 4096, 8192, 8)])
def test_results_in_fp32_fill_the_memorys_time(e, k, n, rows):
    assert _tile(e, k, n, rows, out=B.DT_FLOAT32) == 256


def test_both_types_and_a_given_height():
    assert B.gm_plan(gw(m=32, k=2048, n=2048, e=4, dt=F16, dw=fake(F16, 4, 2048, 2048)))["tile_m"] == 128
    assert _tile(4, 2048, 2048, 8, tuning=[0, 256]) == 256 and _tile(64, 2048, 2048, 64, tuning=[0, 128]) == 128


@pytest.mark.parametrize("side", ["x", "dy"])
@pytest.mark.parametrize("e,k,n", [(8, 2048, 2048), (64, 1536, 2048), (64, 1024, 4096)])
def test_rows_kept_in_fp8_by_the_step(e, k, n, side):
    """One step of 32 rows, and more; results in fp32 by the rounds alone."""
    def tile(rows, out=BF):
        return B.gm_plan(gx(m=e * rows, k=k, n=n, e=e, side=side, dw=fake(out, e, k, n)))["tile_m"]
    assert [tile(r) for r in (1, 32, 33, 64)] == [128, 128, 256, 256]
    assert tile(8, B.DT_FLOAT32) == 256
