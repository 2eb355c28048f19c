"""Clipping where several launches leave more sums than each workgroup adds itself."""
import pytest
import torch

import unstructured_sparse_linear_amd as S
from test_gpu_clip import check, make

pytestmark = pytest.mark.gpu


def sizes(big):
    """A table's 1535, 1536 or 1537 chunks and a second one, of few or of many."""
    return [8192 * big - 250] + [1 + i % 17 for i in range(249)]


@pytest.mark.parametrize("first", [1286, 1287, 1288])  # 249 more chunks in its table
@pytest.mark.parametrize("second", [1, 2, 1500])
def test_two_tables(first, second):
    grads = make(sizes(first) + [8192 * second - 1], "mixed")
    kept = [g.clone() for g in grads]
    outs = [torch.full_like(g, 7.0) for g in grads]
    norm = S.clip_grad_norm(grads, 0.5, out=outs)
    check(grads, outs, norm, 0.5)
    assert torch.equal(norm, S.clip_grad_norm(grads, 0.5))
    for g, o in zip(grads, outs):
        assert torch.equal(g, o)
    below = S.clip_grad_norm(kept, 1e9)  # nothing to change
    assert torch.equal(below, norm)


def test_many_in_a_graph():
    shape = sizes(1400) + sizes(300) + [5]
    grads = make(shape, "bf16")
    outs = [torch.empty_like(g) for g in grads]
    S.clip_grad_norm(grads, 1.0, out=outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = S.clip_grad_norm(grads, 1.0, out=outs)
    for seed in (1, 2, 3):
        for g, n in zip(grads, make(shape, "bf16", seed=seed, std=seed)):
            g.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        check(grads, outs, norm, 1.0)
        eager = [torch.empty_like(g) for g in grads]
        assert torch.equal(norm, S.clip_grad_norm(grads, 1.0, out=eager))
        for a, b in zip(eager, outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("max_norm", [1e9, 0.5])
def test_some_in_place(max_norm):
    """Below the limit what is in place is left alone, and the rest is copied."""
    grads = make([8192 * 1600, 8192 * 1700 + 5, 8192 * 9, 77], "mixed")
    kept = [g.clone() for g in grads]
    outs = [g if i % 2 == 0 else torch.full_like(g, 7.0) for i, g in enumerate(grads)]
    norm = S.clip_grad_norm(grads, max_norm, out=outs)
    check(kept, outs, norm, max_norm)
    assert torch.equal(grads[1], kept[1]) and torch.equal(grads[3], kept[3])
    if max_norm == 1e9:
        for o, k in zip(outs, kept):
            assert torch.equal(o, k)
