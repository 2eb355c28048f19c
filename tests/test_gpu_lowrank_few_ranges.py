"""The one-launch form of a few tokens where u is far outside f16's range, and
where the tokens' ranges lie far apart: each has a scale of its own."""
import pytest
import torch

import unstructured_sparse_linear_amd as S
import lowrank_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("a,b,x", [(1e-3, 1e3, 1e-3), (3e4, 1e-3, 1.0)])
@pytest.mark.parametrize("T,R", [(1, 16), (1, 32), (7, 16), (16, 20)])
def test_few_tokens(T, R, a, b, x):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    c = ref.Case("f16", [T], [1], 2, R, 512, 300)
    c.A.mul_(a)
    c.B.mul_(b)
    c.xt.mul_(x)
    c.yt.mul_(1e-3)
    steps = torch.arange(T, device="cuda")
    c.xt.mul_(torch.pow(2.0, -(steps % 4).float()).to(torch.float16))
    ref.check(S.low_rank_add(c.yt, *c.args()), ref.add(c), "add")
    ref.check(S.low_rank_project(c.W, *c.args()), ref.project(c), "project")
