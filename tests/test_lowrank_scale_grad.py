"""A scale that requires a gradient is refused, not left out."""
import pytest
import torch

import unstructured_sparse_linear_amd as P


def args(scale):
    return (torch.zeros(6, 5), torch.zeros(8, 5), torch.zeros(2, 4, 8), torch.zeros(2, 6, 4),
            torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), scale)


def test_low_rank_linear():
    scale = torch.ones(2, requires_grad=True)
    with pytest.raises(ValueError, match="scale has no gradient"):
        P.low_rank_linear(*args(scale))
    # without it the call goes on to the next check
    with pytest.raises(ValueError, match="GPU tensor"):
        P.low_rank_linear(*args(scale.detach()))
    with torch.no_grad(), pytest.raises(ValueError, match="GPU tensor"):
        P.low_rank_linear(*args(scale))


def test_module():
    for scale in (torch.nn.Parameter(torch.ones(2)),
                  torch.ones(2, dtype=torch.float64, requires_grad=True)):
        m = P.LowRankAdapters(2, 4, 8, 6, scale=scale, device="cpu")
        with pytest.raises(ValueError, match="scale has no gradient"):
            m(*args(None)[:2], *args(None)[4:6])
