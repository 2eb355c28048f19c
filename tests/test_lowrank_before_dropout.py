"""Adapters that were made, or whose class was made, before they had dropout."""
import pytest
import torch

import unstructured_sparse_linear_amd as P
from unstructured_sparse_linear_amd import adapter


@pytest.fixture(autouse=True)
def host(monkeypatch):
    """Stands for the compiled call, which needs a GPU: yt + B A xt of one adapter."""
    monkeypatch.setattr(adapter, "low_rank_linear",
                        lambda yt, xt, A, B, *rest: yt + B[0] @ (A[0] @ xt))


def result(m):
    with torch.no_grad():
        m.B.fill_(1.0)
    return m.train()(torch.zeros(4, 3), torch.ones(4, 3), None, None)


def test_a_module_that_was_kept_whole():
    m = P.LowRankAdapters(1, 2, 4, 4, device="cpu")
    state = m.__dict__.copy()
    del state["dropout"]
    old = P.LowRankAdapters.__new__(P.LowRankAdapters)
    old.__setstate__(state)
    assert old.next_dropout_state() is None
    assert torch.equal(result(old), result(m))


def test_a_class_with_a_layer_of_that_name():
    class Adapters(P.LowRankAdapters):
        def __init__(self, *args, **kw):
            super().__init__(*args, **kw)
            self.dropout = torch.nn.Dropout(0.0)

        def forward(self, yt, xt, offsets, adapter):
            return super().forward(yt, self.dropout(xt), offsets, adapter)

    m = Adapters(1, 2, 4, 4, device="cpu")
    assert isinstance(m.dropout, torch.nn.Dropout) and m.next_dropout_state() is None
    assert torch.equal(result(m), m.B.detach()[0] @ (m.A.detach()[0] @ torch.ones(4, 3)))
