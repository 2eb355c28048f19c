"""Few tokens on both sides of the sizes at which they leave the one-launch form."""
import pytest
import torch

import unstructured_sparse_linear_amd as S
import lowrank_ref as ref

pytestmark = pytest.mark.gpu

SHAPES = {  # tokens, ranks, features in and out; each pair differs by one feature or row
    "add-16": (1, 16, 4608, 272), "add-16-past": (1, 16, 4609, 272),
    "add-32": (16, 32, 2304, 80), "add-32-past": (16, 32, 2305, 80),
    "project-1": (1, 9, 8192, 48), "project-1-past": (1, 9, 8193, 48),
    "project-5": (5, 16, 1024, 4096), "project-5-past": (5, 16, 6145, 40),
    "project-rows": (3, 32, 1024, 8192), "project-rows-past": (3, 32, 1025, 8193),
}


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_edges(shape, dt):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    T, R, n_in, n_out = SHAPES[shape]
    c = ref.Case(dt, [T], [1], 2, R, n_in, n_out)
    ref.check(S.low_rank_add(c.yt, *c.args()), ref.add(c), "add")
    ref.check(S.low_rank_project(c.W, *c.args()), ref.project(c), "project")
