"""The weight gradient of FP8 rows wants a workspace sometimes, and the library
alone says when: the binding keeps no rule of its own (a library that answers,
no GPU needed)."""
import ctypes

import pytest
import torch

from quantized_moe_grouped_amd import binding as B


class Library:
    """Wants `need` bytes whatever the sizes, and notes what it is given."""

    def __init__(self, need, status=B.OK):
        self.need, self.status, self.given = need, status, []

    def gmm_grouped_matmul_wgrad_fp8_workspace(self, raw, out):
        ctypes.cast(out, ctypes.POINTER(ctypes.c_size_t))[0] = self.need
        return B.OK

    def gmm_grouped_matmul_wgrad_fp8(self, raw, workspace, size, stream):
        if self.status == B.OK and size < self.need:
            return B.ERR_WORKSPACE
        self.given.append((workspace, size))
        return self.status


def _call(monkeypatch, library, rows, workspace=None):
    monkeypatch.setattr(B, "_lib", library)
    codes = torch.zeros((rows, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.zeros((rows, 1, 2), dtype=torch.uint8).view(torch.float8_e8m0fnu)
    dy, gl = torch.zeros((rows, 8), dtype=torch.bfloat16), torch.tensor([rows])
    return B._grouped_matmul_wgrad(0, codes, dy, gl, scale, None, None, None, False, 1, None, workspace)


@pytest.mark.parametrize("rows", [1, 2047, 2048, 10000])
def test_one_is_made_where_the_library_wants_it(monkeypatch, rows):
    library = Library(4096)
    assert _call(monkeypatch, library, rows).shape == (1, 64, 8)
    (pointer, size), = library.given
    assert pointer and size == 4096


@pytest.mark.parametrize("rows", [1, 10000])
def test_none_is_made_where_it_wants_none(monkeypatch, rows):
    library = Library(0)
    _call(monkeypatch, library, rows)
    assert library.given == [(0, 0)]


def test_a_given_one_is_passed_on_or_refused(monkeypatch):
    library, own = Library(4096), torch.empty(4096, dtype=torch.uint8)
    _call(monkeypatch, library, 3, own)
    assert library.given == [(own.data_ptr(), 4096)]
    with pytest.raises(B.GmmfrError, match="WORKSPACE"):
        _call(monkeypatch, Library(4096), 3, own[:64])


def test_other_refusals_are_the_callers(monkeypatch):
    library = Library(4096, status=B.ERR_SHAPE)
    with pytest.raises(B.GmmfrError, match="SHAPE"):
        _call(monkeypatch, library, 3)
    assert len(library.given) == 1
