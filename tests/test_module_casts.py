"""Casts and moves of Mx4Linear and of adapters with dropout, on the CPU: whole numbers stay
what they are."""
import copy

import pytest
import torch

import unstructured_sparse_linear_amd as P

CASTS = [lambda m: m.type(torch.bfloat16), lambda m: m.type(torch.float64),
         lambda m: m.to(torch.float16), lambda m: m.half().float(),
         lambda m: torch.nn.Sequential(m).type(torch.bfloat16)[0],
         lambda m: copy.deepcopy(m).type(torch.float16)]


def linear(cols, rows=5, seed=0):
    """A layer with codes of every kind, zeros past the last column."""
    nb = -(-cols // 32)
    g = torch.Generator().manual_seed(seed)
    i = torch.randint(1, 16, (rows, 32 * nb), generator=g)
    i[:, cols:] = 0
    codes = (i[:, 0::2] + 16 * i[:, 1::2]).to(torch.uint8)
    scales = torch.randint(118, 134, (rows, nb), generator=g).to(torch.uint8)
    return P.Mx4Linear(P.Mx4Matrix(codes, scales, cols))


@pytest.mark.parametrize("cast", CASTS)
def test_casts_leave_codes_and_scales(cast):
    m = linear(70)
    want = m.codes.clone(), m.scales.clone()
    m = cast(m)
    assert m.weight.shape == (5, 70)
    assert torch.equal(m.codes, want[0]) and torch.equal(m.scales, want[1])


@pytest.mark.parametrize("cast", CASTS)
def test_casts_leave_the_state_of_dropout(cast):
    scale = torch.tensor([1.0 + 2.0 ** -12, 0.3])
    m = P.LowRankAdapters(2, 4, 8, 6, device="cpu", dropout=0.5, seed=(1 << 60) + 1, scale=scale,
                          ranks=torch.tensor([4, 70_001]))
    m.dropout_state[1] = (1 << 40) + 3
    m = cast(m)
    assert m.dropout_state.dtype == torch.int64
    assert m.dropout_state.tolist() == [(1 << 60) + 1, (1 << 40) + 3]
    assert m.ranks.dtype == torch.int32 and m.ranks.tolist() == [4, 70_001]
    assert m.scale.dtype == torch.float32 and torch.equal(m.scale, scale)


def test_moves_go_on():
    m = linear(70).to("meta")
    assert m.codes.device.type == m.scales.device.type == "meta" and m.codes.dtype == torch.uint8
    m = P.LowRankAdapters(2, 4, 8, 6, device="cpu", dropout=0.5).to("meta", torch.float16)
    assert m.dropout_state.device.type == "meta" and m.A.dtype == torch.float16
