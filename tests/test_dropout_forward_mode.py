"""Dropout of a dual tensor: there is no forward-mode derivative, and the call says so as
the other differentiable ones do, instead of returning a result without its tangent."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import unstructured_sparse_linear_amd as P
from unstructured_sparse_linear_amd import adapter


class OnTheHost:
    """Stands for the compiled binding: writes memory that autograd knows nothing of."""

    @staticmethod
    def dropout(x, p, seed, step, out):
        out = torch.empty(x.shape, dtype=x.dtype) if out is None else out
        out.detach().numpy()[...] = 2 * x.detach().numpy()
        return out


@pytest.fixture
def host(monkeypatch):
    monkeypatch.setattr(adapter, "_marshal", OnTheHost)


def refused(x, **kw):
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        with pytest.raises(NotImplementedError, match="jvp"):
            P.dropout(dual, 0.5, 1, **kw)
        with torch.no_grad(), pytest.raises(NotImplementedError, match="jvp"):
            P.dropout(dual, 0.5, 1, **kw)
        dual = fwd.make_dual(x.clone().requires_grad_(), torch.ones_like(x))
        with pytest.raises(NotImplementedError, match="jvp"):
            P.dropout(dual, 0.5, 1, **kw)


def refused_into_out(x):
    with fwd.dual_level():
        dual, out = fwd.make_dual(x, torch.ones_like(x)), torch.full_like(x, 7.0)
        with torch.no_grad(), pytest.raises(ValueError, match="no gradient"):
            P.dropout(dual, 0.5, 1, out=out)
        with pytest.raises(ValueError, match="no gradient"):
            P.dropout(x, 0.5, 1, out=fwd.make_dual(out, torch.ones_like(x)))
        assert (out == 7.0).all()


def test_dual_tensor(host):
    refused(torch.ones(3, 8))


def test_dual_tensor_into_out(host):
    refused_into_out(torch.ones(3, 8))


def test_others_at_a_dual_level(host):
    """What has no tangent is computed as it is elsewhere."""
    x = torch.ones(3, 8)
    with fwd.dual_level():
        assert torch.equal(P.dropout(x, 0.5, 1), 2 * x)
        assert P.dropout(x, 0.5, 1, out=x) is x


@pytest.mark.gpu
def test_dual_tensor_on_the_gpu():
    x = torch.ones(3, 8, device="cuda")
    refused(x)
    refused_into_out(x)
    layer = P.LowRankAdapters(1, 2, 3, 3, dropout=0.5, seed=1)
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    which = torch.zeros(1, dtype=torch.int32, device="cuda")
    with fwd.dual_level(), pytest.raises(NotImplementedError, match="jvp"):
        layer(torch.zeros_like(x), fwd.make_dual(x, x), off, which)
