"""Refusals of clip_grad_norm where outputs would be written twice or over other
gradients, without a GPU (a call that passes them is refused for its device)."""
import pytest
import torch

import unstructured_sparse_linear_amd as P

OWN = "must be a tensor of its own"
NEXT = "must be a GPU tensor"


def test_a_tensor_twice():
    a, b = torch.zeros(4), torch.zeros(5)
    for grads in ([a, a], [a, b, a], [a, b, b[:3]], [a, a.view(2, 2)]):
        with pytest.raises(ValueError, match="every gradient " + OWN):
            P.clip_grad_norm(grads, 1.0)
        outs = [torch.zeros_like(g) for g in grads]
        with pytest.raises(ValueError, match=NEXT):  # read twice, written once each
            P.clip_grad_norm(grads, 1.0, out=outs)
    many = [torch.zeros(1 + i % 3) for i in range(700)]
    with pytest.raises(ValueError, match=NEXT):
        P.clip_grad_norm(many, 1.0)
    with pytest.raises(ValueError, match=OWN):
        P.clip_grad_norm(many + many[123:124], 1.0)


def test_outputs():
    a, b, c = torch.zeros(4), torch.zeros(4), torch.zeros(4)
    for outs in ([c, c], [b, a], [a, a], [b, c], [c, a]):
        with pytest.raises(ValueError, match="every out " + OWN):
            P.clip_grad_norm([a, b], 1.0, out=outs)
    for outs in ([a, b], [c, b], [a, c], [c, torch.zeros(4)]):
        with pytest.raises(ValueError, match=NEXT):
            P.clip_grad_norm([a, b], 1.0, out=outs)


def test_tensors_without_values_may_repeat():
    e, a = torch.zeros(0), torch.zeros(3)
    with pytest.raises(ValueError, match=NEXT):
        P.clip_grad_norm([e, a, e, torch.zeros(0)], 1.0)
