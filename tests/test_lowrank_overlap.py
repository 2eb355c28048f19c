"""Workspace of low-rank adapter calls whose out shares memory with xt, without
a GPU (no pointer below is dereferenced: every call is refused)."""
import ctypes

import pytest

import unstructured_sparse_linear_amd.spops as S
from test_lowrank_refusals import FAKE, L, desc, need  # noqa: F401

ADD, PROJECT, BACKWARD, OVER_X = 0, 1, 2, 4


def square(**kw):
    return desc(**{**dict(tokens=8, requests=1, in_features=64, out_features=64), **kw})


def test_workspace_size(L):  # noqa: F811
    for op in (ADD, PROJECT):
        assert need(L, square(), op) == 0  # one launch
        assert need(L, square(), op | OVER_X) >= 16 * 8 * 4  # u between two
        assert need(L, square(tokens=40), op | OVER_X) == need(L, square(tokens=40), op)
        assert need(L, square(tokens=0), op | OVER_X) == 0
    b = ctypes.c_size_t()
    for op in (BACKWARD | OVER_X, 3 | OVER_X, 8, -1):
        assert L.spops_low_rank_workspace_size(ctypes.byref(square()), op, ctypes.byref(b)) == 6


@pytest.mark.parametrize("op", [ADD, PROJECT])
@pytest.mark.parametrize("shift", [0, 2, -2, 64 * 16 - 2, 2 - 64 * 16])
def test_few_tokens_over_x_need_it(L, op, shift):  # noqa: F811
    """Up to 16 tokens run in one launch that reads all of xt while it writes
    out: not where the two share memory."""
    f = L.spops_low_rank_project if op == PROJECT else L.spops_low_rank_add
    lead = 64 if op == PROJECT else 8
    big = need(L, square(), op | OVER_X)
    first = FAKE << 8
    for ws, size in ((None, 0), (FAKE, big - 1), (FAKE + 16, big)):
        assert f(ctypes.byref(square()), first, lead, FAKE, 8, FAKE + shift, 8, ws, size,
                 None) == 5
