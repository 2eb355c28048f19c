"""Which calls of few tokens run in one launch (and so need no workspace): those
whose workgroups read little for themselves."""
import pytest

from test_lowrank_refusals import L, desc, need  # noqa: F401

ADD, PROJECT = 0, 1
F32, F16, BF16 = 0, 1, 2


def one_launch(L, op, n_in, n_out, rank, tokens=1, dtype=BF16, requests=1):  # noqa: F811
    return need(L, desc(tokens=tokens, requests=requests, adapters=8, rank=rank, in_features=n_in,
                        out_features=n_out, dtype=dtype), op) == 0


@pytest.mark.parametrize("n_in,rank,dtype,one", [
    (4096, 16, BF16, True), (4096, 3, F16, True), (4608, 16, BF16, True), (4609, 16, BF16, False),
    (11008, 16, BF16, False), (2304, 32, F16, True), (4096, 32, BF16, False),
    (2304, 16, F32, True), (4096, 16, F32, False), (1024, 33, BF16, False)])
def test_add(L, n_in, rank, dtype, one):  # noqa: F811
    for n_out in (16, 4096, 16384):
        for tokens in (1, 16):
            assert one_launch(L, ADD, n_in, n_out, rank, tokens, dtype) == one
        assert not one_launch(L, ADD, n_in, n_out, rank, 17, dtype)
        assert not one_launch(L, ADD, n_in, n_out, rank, 16, dtype, requests=2)


@pytest.mark.parametrize("n_in,n_out,rank,tokens,one", [
    (4096, 4096, 16, 1, True), (4096, 4096, 16, 16, True), (4096, 4096, 32, 16, True),
    (8192, 4096, 16, 1, True), (8192, 4096, 16, 2, False), (8192, 4096, 32, 1, False),
    (4096, 11008, 16, 1, False), (1024, 11008, 16, 1, True), (1024, 11008, 32, 2, True),
    (2048, 11008, 16, 2, False), (4096, 16384, 16, 1, True), (4096, 16384, 16, 2, False),
    (11008, 4096, 16, 1, False), (65536, 1024, 16, 1, False)])
def test_project(L, n_in, n_out, rank, tokens, one):  # noqa: F811
    assert one_launch(L, PROJECT, n_in, n_out, rank, tokens) == one
