"""Which tile the plans of the gated block, its way back and the weight gradients
take, on both sides of every bound (host only, fake pointers)."""
import ctypes

import pytest

from quantized_moe_grouped_amd import binding as B
from tests.test_boundary_gated import gb, gf, gx, in_fp8
from tests.test_boundary_grouped import BF, fake, gm, gw


def _gf(m, f, e=1, k=512, turned=False, fp8=False, **over):
    if turned:
        over.update(transpose_w=1, w=fake(BF, e, 2 * f, k))
    if fp8:
        over.update(in_fp8(m, f))
    return gf(m=m, k=k, f=f, e=e, **over)


def _gb(m, f, e=1, k=512, turned=True, fp8=False, **over):
    if not turned:
        over.update(transpose_w=0, w=fake(BF, e, k, f))
    if fp8:
        over.update(in_fp8(m, f))
    return gb(m=m, k=k, f=f, e=e, **over)


def _tile(args):
    p = B.gm_plan(args)
    return p["tile_m"], p["tile_n"]


@pytest.mark.parametrize("make,sizes,tile", [
    # narrow tiles of 64 columns: one round of 512 workgroups, two with weights (e,n,k); 64 rows are two of them
    (_gf, dict(m=64, f=8192), (32, 64)), (_gf, dict(m=64, f=8224), (128, 128)),
    (_gf, dict(m=64, f=16384, turned=True), (32, 64)), (_gf, dict(m=64, f=16416, turned=True), (128, 128)),
    (_gf, dict(m=64, f=8192, fp8=True), (32, 64)), (_gf, dict(m=64, f=8224, fp8=True), (128, 128)),
    (_gb, dict(m=128, f=8192, turned=False), (32, 64)), (_gb, dict(m=128, f=8200, turned=False), (128, 128)),
    (_gb, dict(m=128, f=16384), (32, 64)), (_gb, dict(m=128, f=16416, fp8=True), (128, 128)),
    # several experts: by the rows that each has on average
    (_gf, dict(m=8 * 40, e=8, f=1024), (32, 64)), (_gf, dict(m=8 * 40, e=8, f=1032), (128, 128)),
    (_gf, dict(m=8 * 40, e=8, f=2048, turned=True), (32, 64)), (_gf, dict(m=8 * 40, e=8, f=2056, turned=True), (128, 128)),
    # 32 columns: weights (e,n,k) under 256 tiles of 64 and fewer, and never where a scale's 32 columns are kept in FP8
    (_gf, dict(m=64, f=2720, turned=True), (32, 32)), (_gf, dict(m=64, f=2752, turned=True), (32, 64)),
    (_gf, dict(m=64, f=2720, turned=True, fp8=True), (32, 64)), (_gf, dict(m=64, f=2720), (32, 64)),
    (_gf, dict(m=1, f=4096, turned=True), (32, 32)), (_gf, dict(m=1, f=4096, turned=True, fp8=True), (32, 64)),
    (_gb, dict(m=64, f=5440), (32, 32)), (_gb, dict(m=64, f=5440, fp8=True), (32, 32)), (_gb, dict(m=64, f=5472, fp8=True), (32, 64)),
    (_gb, dict(m=64, f=5440, turned=False), (32, 64)),
    # many rows: by the rounds that the larger tiles make
    (_gf, dict(m=4096, f=2048), (256, 256)), (_gf, dict(m=4096, f=1024), (128, 128)),
    (_gb, dict(m=4096, f=2048), (128, 128)), (_gb, dict(m=8192, f=2048), (256, 256)),
])
def test_the_tile_taken(make, sizes, tile):
    assert _tile(make(**sizes)) == tile


def test_the_plain_product_keeps_its_own_rules():
    """The same product without a gate stays on the 128-row tiles there."""
    assert _tile(gm(m=64, k=512, n=16384, e=1)) == (128, 128)
    assert _tile(_gf(64, 8192)) == (32, 64)


@pytest.mark.parametrize("height", [32, 128, 256])
def test_a_given_height_is_taken(height):
    for args in (_gf(64, 8192, tuning=[0, height]), _gb(4096, 2048, tuning=[0, height])):
        assert _tile(args)[0] == height


def test_expected_rows():
    """One of eight experts has them all: whole tiles of that many."""
    assert _tile(_gf(2048, 2048, e=8)) == (256, 256)
    assert _tile(_gf(2048, 2048, e=8, tuning=[16])) == (32, 64)
    assert _tile(_gf(4096, 2048, e=8, tuning=[4096])) == (256, 256)


@pytest.mark.parametrize("args,tile", [
    (gw(m=32768, k=2048, n=7168, e=32), (256, 256)), (gw(m=300, k=512, n=384, e=4), (128, 128)),
    (gx(m=32768, k=7168, n=4096, e=32), (256, 256)), (gx(m=6007, k=1088, n=1600, e=48), (128, 128)),
    # split rows: 256-row tiles where their parts fill three quarters of the chip
    (gx(m=16384, k=2048, n=2048, e=1), (256, 256)), (gx(m=8192, k=512, n=512, e=1), (128, 128)),
    (gx(m=16384, k=1024, n=1024, e=1, side="dy"), (256, 256)), (gx(m=16384, k=512, n=512, e=4), (128, 128)),
])
def test_weight_gradients(args, tile):
    assert _tile(args) == tile


def test_plans_refuse_as_the_calls_do():
    info = B.GmPlanInfo()
    for name, make, bad in (("gmm_gated_matmul", _gf, dict(m=64, f=36)), ("gmm_gated_matmul_backward", _gb, dict(m=64, f=36)),
                            ("gmm_grouped_matmul_wgrad", gw, dict(n=12)), ("gmm_grouped_matmul_wgrad_fp8", gx, dict(n=12))):
        plan = getattr(B.lib(), name + "_plan")
        good = make(**{**bad, "f": 64}) if "f" in bad else make()
        assert plan(ctypes.byref(make(**bad)), ctypes.byref(info)) == B.ERR_SHAPE
        assert plan(None, ctypes.byref(info)) == B.ERR_NULLPTR and plan(ctypes.byref(good), None) == B.ERR_NULLPTR
        assert plan(ctypes.byref(good), ctypes.byref(info)) == B.OK and info.grid > 0
    for args in (_gf(0, 64), _gb(0, 64)):  # nothing to launch
        assert B.gm_plan(args)["grid"] == 0
    assert B.gm_plan(gw(m=0))["grid"] > 0  # zeros are written
