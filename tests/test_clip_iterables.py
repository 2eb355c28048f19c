"""clip_grad_norm takes its tensors from any iterable, without a GPU (a call that
passes the checks of its tensors is refused for their device)."""
import pytest
import torch

import unstructured_sparse_linear_amd as P


@pytest.mark.parametrize("as_given", [list, tuple, iter, lambda t: (x for x in t),
                                      lambda t: dict(enumerate(t)).values()])
def test_iterables(as_given):
    grads = [torch.zeros(4), torch.zeros(3, dtype=torch.bfloat16)]
    outs = [torch.zeros(4), torch.zeros(3, dtype=torch.bfloat16)]
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        P.clip_grad_norm(as_given(grads), 1.0)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        P.clip_grad_norm(as_given(grads), 1.0, out=as_given(outs))
    with pytest.raises(ValueError, match="at least one tensor"):
        P.clip_grad_norm(as_given([]), 1.0)
