"""What autograd of the low-rank adapters refuses instead of leaving out."""
import pytest
import torch

import unstructured_sparse_linear_amd as S
import lowrank_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    S.lib()
    yield
    torch.cuda.synchronize()


def case():
    return ref.Case("f32", [20, 13], [1, 0], 2, 8, 96, 80)


@pytest.mark.parametrize("name", ["xt", "A", "B"])
def test_second_derivatives_raise(name):
    """The gradient's own graph has no adapters' part: using it is an error."""
    c = case()
    t = getattr(c, name).requires_grad_()
    w = torch.ones((), device="cuda", requires_grad=True)
    y = S.low_rank_linear(c.yt, *c.args())
    grad, = torch.autograd.grad((w * y * y).sum(), t, create_graph=True)
    want = torch.autograd.grad((y.detach() * y).sum() * 2, t, retain_graph=False)[0]
    assert torch.allclose(grad, want, rtol=1e-5, atol=1e-5)  # the first one is there
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.square().sum().backward()
