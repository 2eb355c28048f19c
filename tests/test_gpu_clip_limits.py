"""Gradient clipping without a limit: the norm alone."""
import pytest
import torch

import unstructured_sparse_linear_amd as S
from test_gpu_clip import make

pytestmark = pytest.mark.gpu
INF = float("inf")


def same(a, b):
    return torch.equal(a.nan_to_num(7.0, 8.0, 9.0), b.nan_to_num(7.0, 8.0, 9.0))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16", "mixed"])
@pytest.mark.parametrize("bad", [INF, -INF, float("nan"), None])
def test_an_infinite_limit_changes_nothing(dt, bad):
    grads = make([5, 9000, 8192, 16_384], dt)
    if bad is not None:
        grads[1][77] = bad
        grads[2][0] = bad
    kept = [g.clone() for g in grads]
    outs = [torch.zeros_like(g) for g in grads]
    for norm in (S.clip_grad_norm(grads, INF, out=outs), S.clip_grad_norm(grads, INF)):
        if bad is None:
            assert norm.isfinite()
        else:
            assert norm.isnan() if bad != bad else norm == INF
    for g, o, k in zip(grads, outs, kept):
        assert same(g, k) and same(o, k)
        assert g.isfinite().sum() >= g.numel() - 1
