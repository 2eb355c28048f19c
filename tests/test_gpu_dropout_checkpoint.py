"""Adapters with dropout whose forward pass is run again in the backward pass
(torch.utils.checkpoint): the same mask where the state is given, a refusal where
another one would be drawn."""
import pytest
import torch
from torch.utils.checkpoint import checkpoint

import unstructured_sparse_linear_amd as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    S.lib()
    yield
    torch.cuda.synchronize()


class Block:
    """A frozen 4-bit layer, adapters on it, and a batch of two requests."""

    def __init__(self, seed=5, **kw):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.base = S.Mx4Linear(torch.randn(50, 60, generator=g, device="cuda"))
        self.layer = S.LowRankAdapters(2, 4, 60, 50, dropout=0.5, seed=seed, **kw)
        with torch.no_grad():
            for factor in (self.layer.A, self.layer.B):
                factor.normal_(generator=g)
        self.xt = torch.randn(60, 20, generator=g, device="cuda", requires_grad=True)
        self.dy = torch.randn(50, 20, generator=g, device="cuda")
        self.off = torch.tensor([0, 7, 20], dtype=torch.int32, device="cuda")
        self.which = torch.tensor([1, 0], dtype=torch.int32, device="cuda")

    def __call__(self, xt, *state):
        return self.layer(self.base(xt), xt, self.off, self.which, *state)

    def inputs(self):
        return self.xt, self.layer.A, self.layer.B

    def step(self):
        """Result and gradients of one step without recomputation."""
        y = self(self.xt)
        return [y.detach(), *torch.autograd.grad(y, self.inputs(), self.dy)]

    def backward(self, y):
        for t in self.inputs():
            t.grad = None
        y.backward(self.dy)
        return [y.detach(), *(t.grad for t in self.inputs())]


MODES = [False, True]


@pytest.mark.parametrize("reentrant", MODES)
def test_gradients_with_a_given_state(reentrant):
    a, b = Block(), Block()
    for i in range(3):
        want = a.step()
        state = b.layer.next_dropout_state()
        assert state.tolist() == [5, i] and b.layer.dropout_state.tolist() == [5, i + 1]
        got = b.backward(checkpoint(b, b.xt, state, use_reentrant=reentrant))
        assert all(torch.equal(x, y) for x, y in zip(got, want)), i
        assert b.layer.dropout_state.tolist() == [5, i + 1]


@pytest.mark.parametrize("reentrant", MODES)
def test_a_new_mask_in_the_backward_pass_is_refused(reentrant):
    b = Block()
    y = checkpoint(b, b.xt, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="next_dropout_state"):
        b.backward(y)
    assert b.layer.dropout_state.tolist() == [5, 1]
    # so is one that is drawn in there by hand
    y = checkpoint(lambda xt: b(xt, b.layer.next_dropout_state()), b.xt, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="next_dropout_state"):
        b.backward(y)
    assert b.layer.dropout_state.tolist() == [5, 2]
    # and the module is as good as before
    a = Block()
    a.layer.dropout_state.copy_(b.layer.dropout_state)
    assert all(torch.equal(x, y) for x, y in zip(b.step(), a.step()))


@pytest.mark.parametrize("reentrant", MODES)
def test_a_state_restored_by_hand(reentrant):
    a, b = Block(), Block()
    want = a.step()
    first = b.layer.dropout_state.clone()

    def again(xt):
        b.layer.dropout_state.copy_(first)
        return b(xt)

    got = b.backward(checkpoint(again, b.xt, use_reentrant=reentrant))
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert b.layer.dropout_state.tolist() == [5, 1]


@pytest.mark.parametrize("reentrant", MODES)
def test_without_dropout_nothing_is_refused(reentrant):
    a, b = Block(), Block()
    for blocks in (a, b):
        blocks.layer.eval()
    want = a.step()
    assert b.layer.next_dropout_state() is None
    got = b.backward(checkpoint(b, b.xt, b.layer.next_dropout_state(), use_reentrant=reentrant))
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    got = b.backward(checkpoint(b, b.xt, use_reentrant=reentrant))
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert b.layer.dropout_state.tolist() == [5, 0]


def test_two_blocks_run_again():
    """Several layers between two kept activations, each with a state of its own."""
    blocks = [Block(5), Block(6)]
    blocks[1].base = S.Mx4Linear(torch.randn(60, 50, device="cuda"))
    second = S.LowRankAdapters(2, 4, 50, 60, dropout=0.25, seed=6)
    with torch.no_grad():
        second.B.normal_()
    blocks[1].layer = second

    def both(xt, *states):
        for i, block in enumerate(blocks):
            xt = block(xt, *states[i:i + 1])
        return xt

    xt = blocks[0].xt
    leaves = [xt, *(p for b in blocks for p in b.layer.parameters())]
    want = torch.autograd.grad(both(xt).sum(), leaves)
    for b in blocks:
        b.layer.dropout_state[1].zero_()
    y = checkpoint(both, xt, *(b.layer.next_dropout_state() for b in blocks), use_reentrant=False)
    got = torch.autograd.grad(y.sum(), leaves)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert [b.layer.dropout_state.tolist() for b in blocks] == [[5, 1], [6, 1]]


def test_captured_with_a_given_state():
    """A state taken inside a captured step is another one at each replay."""
    b = Block()

    def step():
        y = b(b.xt, b.layer.next_dropout_state())
        return [y.detach(), *torch.autograd.grad(y, b.inputs(), b.dy)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    a = Block()
    for i in range(3):
        a.layer.dropout_state.copy_(b.layer.dropout_state)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, a.step())), i
        assert torch.equal(a.layer.dropout_state, b.layer.dropout_state)


def test_states_that_are_refused():
    b = Block()
    for state in (torch.zeros(3, dtype=torch.int64, device="cuda"), torch.zeros(2, device="cuda")):
        with pytest.raises(ValueError, match="int64 vector"):
            b(b.xt, state)
    with pytest.raises(ValueError, match="GPU tensor"):
        b(b.xt, torch.zeros(2, dtype=torch.int64))
    assert b.layer.dropout_state.tolist() == [5, 0]
