"""Second derivatives of the sparse layer raise: its gradients have no graph."""
import pytest
import torch

import unstructured_sparse_linear_amd as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("by", ["values", "xt"])
def test_second_derivatives_raise(by):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    offsets = torch.tensor([0, 2, 3, 4], dtype=torch.int32, device="cuda")
    columns = torch.tensor([0, 3, 1, 2], dtype=torch.int32, device="cuda")
    pattern = S.SparsePattern(offsets, columns, 3, 4)
    values = torch.tensor([1.0, 2.0, -1.0, 3.0], device="cuda", requires_grad=True)
    xt = torch.arange(8.0, device="cuda").reshape(4, 2).requires_grad_()
    t = {"values": values, "xt": xt}[by]
    y = S.sparse_linear(values, xt, pattern)
    grad, = torch.autograd.grad(y.square().sum(), t, create_graph=True)
    assert grad.count_nonzero() > 0
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.square().sum().backward()
