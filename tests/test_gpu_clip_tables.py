"""Clipping of more tensors than one launch's table holds, in f64 sums."""
import pytest
import torch

import unstructured_sparse_linear_amd as S
from test_gpu_clip import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [249, 250, 251, 500, 501, 1003])
@pytest.mark.parametrize("empty", [0, 3])
def test_tables(count, empty):
    """Tables that are full, one over, and tensors without values among them."""
    sizes = [0 if empty and i % empty == 0 else 1 + (37 * i) % 190 for i in range(count)]
    sizes[count // 2] = 20_011
    grads = make(sizes, "mixed")
    outs = [torch.full_like(g, 7.0) for g in grads]
    check(grads, outs, S.clip_grad_norm(grads, 0.5, out=outs), 0.5)


@pytest.mark.parametrize("chunks", [1535, 1536, 1537, 6143, 6144, 6145])
def test_launch_widths(chunks):
    """Around the numbers of workgroups at which the launch changes."""
    grads = make([8192 * chunks - 5, 3], "bf16")
    outs = [torch.empty_like(g) for g in grads]
    check(grads, outs, S.clip_grad_norm(grads, 1.0, out=outs), 1.0)
