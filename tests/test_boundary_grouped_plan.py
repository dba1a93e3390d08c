"""Stage one of the grouped products on the CPU: what it says of the workspace."""
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
