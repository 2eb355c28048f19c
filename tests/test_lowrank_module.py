"""LowRankAdapters' buffers on the CPU: what the constructor makes of them, and
what moves and casts of the module leave."""
import copy

import pytest
import torch

import unstructured_sparse_linear_amd as P

SCALE = torch.tensor([1.0 + 2.0 ** -12, 0.3, 70_000.0])  # none is a 16-bit value


def module(**kw):
    kw = {"scale": SCALE, "ranks": torch.tensor([4, 2, 0], dtype=torch.int32), **kw}
    return P.LowRankAdapters(3, 4, 8, 6, device="cpu", **kw)


@pytest.mark.parametrize("cast", [
    lambda m: m.to(torch.bfloat16), lambda m: m.half(), lambda m: m.bfloat16(),
    lambda m: m.to("cpu", torch.float16), lambda m: m.half().float(),
    lambda m: torch.nn.Sequential(m).to(torch.bfloat16)[0],
    lambda m: copy.deepcopy(m).bfloat16()])
def test_casts_leave_scale_and_ranks(cast):
    m = cast(module())
    assert m.scale.dtype == torch.float32 and torch.equal(m.scale, SCALE)
    assert m.ranks.dtype == torch.int32 and m.ranks.tolist() == [4, 2, 0]
    assert m.A.dtype == m.B.dtype


def test_casts_reach_the_factors():
    assert module().to(torch.bfloat16).A.dtype == torch.bfloat16
    assert module(scale=None, ranks=None).half().B.dtype == torch.float16


def test_moves():
    m = module().to("meta")
    assert m.scale.device.type == "meta" and m.scale.dtype == torch.float32
    m = module().to("meta", torch.bfloat16)
    assert m.scale.device.type == "meta" and m.scale.dtype == torch.float32
    m = P.LowRankAdapters(3, 4, 8, 6, scale=SCALE, ranks=torch.tensor([4, 2, 0]), device="meta")
    assert m.scale.device.type == m.ranks.device.type == m.A.device.type == "meta"


def test_types_given():
    m = module(scale=SCALE.double(), ranks=torch.tensor([4, 2, 0]))
    assert m.scale.dtype == torch.float32 and torch.equal(m.scale, SCALE)
    assert m.ranks.dtype == torch.int32
    assert set(m.state_dict()) == {"A", "B", "scale", "ranks"}


def test_state_dict_round_trip():
    m, n = module(), module(scale=torch.ones(3))
    n.load_state_dict(m.bfloat16().state_dict())
    assert torch.equal(n.scale, SCALE) and n.scale.dtype == torch.float32
