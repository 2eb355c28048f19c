"""Sizes whose workgroups an int does not count are refused before the workspace
is looked at, without a GPU; those just below go on to that check."""
import ctypes

import pytest

from test_lowrank_refusals import FAKE, L, desc  # noqa: F401

ADD, PROJECT, BACKWARD = 0, 1, 2
SHAPE, WORKSPACE = 2, 5


def call(L, op, d, lead):  # noqa: F811
    f = getattr(L, "spops_low_rank_" + ("add", "project", "backward")[op])
    grads = (FAKE, FAKE) if op == BACKWARD else ()
    return f(ctypes.byref(d), FAKE, lead, FAKE, d.tokens, FAKE << 24, d.tokens, *grads, None, 0,
             None)


@pytest.mark.parametrize("op", [ADD, PROJECT, BACKWARD])
def test_shrink_blocks(L, op):  # noqa: F811
    """2^24 tiles of four tokens a lane, 64 groups of adapters, blocks of 64 ranks."""
    big = dict(tokens=1 << 30, requests=2 ** 31 - 2, adapters=65535, in_features=16,
               out_features=16)
    lead = 16 if op == PROJECT else 1 << 30
    assert call(L, op, desc(rank=256, **big), lead) == SHAPE
    assert call(L, op, desc(rank=33, **big), lead) == (SHAPE if op == BACKWARD else WORKSPACE)
    assert call(L, op, desc(rank=33, **{**big, "tokens": 1 << 20}), 1 << 20) == WORKSPACE


@pytest.mark.parametrize("op", [ADD, PROJECT, BACKWARD])
def test_tiles(L, op):  # noqa: F811
    for tokens, out, code in ((1 << 20, 1 << 18, WORKSPACE), (1 << 20, 1 << 19, SHAPE)):
        d = desc(tokens=tokens, out_features=out, requests=1)
        assert call(L, op, d, max(tokens, 64)) == code


def test_pool(L):  # noqa: F811
    for n_in, code in ((1 << 18, WORKSPACE), (1 << 21, SHAPE)):
        d = desc(tokens=40, adapters=65535, rank=1, in_features=n_in, out_features=16, requests=1)
        assert call(L, BACKWARD, d, 40) == code
