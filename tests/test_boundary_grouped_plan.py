"""Stage one of the grouped products on the CPU: what it says of the workspace,
and which tile the plan takes under expected rows."""
import ctypes

import pytest

from quantized_moe_grouped_amd import binding as B
from tests import test_boundary_grouped as T


@pytest.mark.parametrize("name,args", [
    ("gmm_grouped_matmul", T.gm()), ("gmm_grouped_matmul", T.gm(e=1024)), ("gmm_grouped_matmul", T.gm(m=0)),
    ("gmm_grouped_matmul", T.mx()), ("gmm_grouped_matmul", T.mx(xt=T.FP8, activation=1, y=T.fake(T.BF, 300, 192))),
    ("gmm_grouped_matmul_wgrad", T.gw()), ("gmm_grouped_matmul_wgrad", T.gw(e=1024, accumulate=1)),
])
def test_no_workspace_is_wanted(name, args):
    assert T.stage_one(name, args) == (B.OK, 0)


@pytest.mark.parametrize("name,args", [("gmm_grouped_matmul", T.gm(m=0)), ("gmm_grouped_matmul", T.mx(m=0))])
def test_none_is_asked_for_in_stage_two(name, args):
    """Without rows nothing is launched: stage two's answer without a workspace, on the CPU."""
    assert getattr(B.lib(), name)(ctypes.byref(args), None, 0, None) == B.OK


def _tile(make=T.gm, rows=None, height=0, cap=0, **sizes):
    tuning = {} if rows is None else dict(tuning=[rows, height, cap])
    return B.gm_plan(make(**sizes, **tuning))


SPREAD = dict(m=8192, e=256, k=2048, n=7168)      # 32 rows an expert, if all have some
CAPACITY = dict(m=32768, e=32, k=2048, n=7168)    # 1024


def test_expected_rows_say_how_many_experts_are_busy():
    assert _tile(**SPREAD)["tile_m"] == 128
    assert _tile(rows=0, **SPREAD)["tile_m"] == 128
    assert _tile(rows=1024, **SPREAD)["tile_m"] == 256   # eight of them have all rows
    assert _tile(rows=256, **SPREAD)["tile_m"] == 256
    assert _tile(rows=8192, **SPREAD)["tile_m"] == 256   # one has
    assert _tile(rows=2 ** 62, **SPREAD)["tile_m"] == 256
    assert _tile(rows=32, **SPREAD) == _tile(**SPREAD)   # what is taken without


def test_expected_rows_of_a_batch_that_is_mostly_spare():
    assert _tile(**CAPACITY)["tile_m"] == 256
    assert _tile(rows=1024, **CAPACITY) == _tile(**CAPACITY)
    assert _tile(rows=150, **CAPACITY)["tile_m"] == 256
    assert _tile(rows=40, **CAPACITY)["tile_m"] == 128
    assert _tile(T.mx, rows=4, **CAPACITY)["tile_m"] == 32
    assert _tile(T.mx, **CAPACITY)["tile_m"] == 256


@pytest.mark.parametrize("make", [T.gm, T.mx])
@pytest.mark.parametrize("rows", [0, 1, 16, 17, 33, 1000, 2 ** 31, 2 ** 63 - 1])
def test_any_expected_rows_make_a_plan(make, rows):
    """The launch holds every tile there may be: it is not sized by what is expected."""
    for sizes in (dict(m=1), dict(m=0), dict(m=2 ** 31 - 1, n=256, e=1024), SPREAD, CAPACITY):
        plan = _tile(make, rows=rows, **sizes)
        assert plan["tile_m"] in (32, 128, 256) and plan["grid"] <= 512
        assert (plan["grid"] == 0) == (sizes["m"] == 0)
        if sizes["m"] > 1:
            assert plan["grid"] == 256 * (1 if plan["tile_m"] == 256 else 2)


def test_a_forced_height_and_a_cap_are_kept():
    for height in (32, 128, 256):
        for rows in (0, 5, 4096):
            plan = _tile(rows=rows, height=height, cap=24, **SPREAD)
            assert (plan["tile_m"], plan["grid"]) == (height, 24)


def test_the_plan_refuses_as_stage_one_does():
    with pytest.raises(B.GmmfrError, match="SHAPE"):
        B.gm_plan(T.gm(k=12))
    assert B.lib().gmm_grouped_matmul_plan(ctypes.byref(T.gm()), None) == B.ERR_NULLPTR
