"""Infinities in the operands of the low-rank adapter calls give what the
definition gives: an infinity times a value of either sign, however many parts
the kernels split the value into; NaN only for infinity times zero and for the
sum of opposite infinities.  Inputs are small integers, so that every sum is
exact in fp32 and each output is the definition's value rounded once."""
import pytest
import torch

import unstructured_sparse_linear_amd as S
import lowrank_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "f16", "bf16"]
INF = float("inf")

SHAPES = {  # lengths, adapter, pool, rank
    "one-token": ([1], [0], 1, 16),
    "few-32-ranks": ([9], [1], 2, 32),
    "decode": ([1] * 20, [i % 3 for i in range(20)], 3, 16),
    "decode-33-ranks": ([1] * 40, [i % 5 - 1 for i in range(40)], 4, 33),
    "prompts": ([100, 37, 131], [1, 0, 1], 2, 7),
    "prompts-24-ranks": ([200, 37, 31], [1, 0, 1], 2, 24),
    "prompts-64-ranks": ([210], [0], 1, 64),
    "prompts-100-ranks": ([130, 70], [0, 1], 2, 100),
}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    S.lib()
    yield
    torch.cuda.synchronize()


def integers(dt, lengths, adapter, n, R, n_in=24, n_out=40):
    c = ref.Case(dt, lengths, adapter, n, R, n_in, n_out)
    g = torch.Generator().manual_seed(5)
    for name, most in (("A", 2), ("B", 3), ("xt", 2), ("yt", 50), ("dyt", 2), ("W", 3)):
        t = getattr(c, name)
        t.copy_(torch.randint(-most, most + 1, t.shape, generator=g))
    c.scale = torch.tensor([0.5, 1.0, 2.0, 1.0][:n], device="cuda")
    return c


def product(a, b):
    """a b in float64, term by term."""
    return (a[:, :, None] * b[None, :, :]).sum(1)


def definition(c):
    """(add, project, dx, dA, dB) request by request, on the CPU."""
    at = {k: getattr(c, k).double().cpu() for k in ("A", "B", "xt", "yt", "dyt", "W")}
    add, project = at["yt"].clone(), product(at["W"], at["xt"])
    dx, dA, dB = torch.zeros_like(at["xt"]), torch.zeros_like(at["A"]), torch.zeros_like(at["B"])
    for t, a, k, s in c.runs():
        x, dy, A, B = at["xt"][:, t], at["dyt"][:, t], at["A"][a, :k], at["B"][a, :, :k]
        u, du = s * product(A, x), s * product(B.t(), dy)
        y = product(B, u)
        add[:, t] += y
        project[:, t] += y
        dx[:, t] = product(A.t(), du)
        dA[a, :k] += product(du, x.t())
        dB[a, :, :k] += product(dy, u.t())
    return add, project, dx, dA, dB


def results(c):
    return (S.low_rank_add(c.yt, *c.args()), S.low_rank_project(c.W, *c.args()),
            *S.low_rank_backward(c.dyt, *c.args()))


NAMES = ("add", "project", "dx", "dA", "dB")


def check_equal(c):
    for name, got, want in zip(NAMES, results(c), definition(c)):
        want = want.to(got.dtype)
        got = got.cpu()
        wrong = ~((got == want) | (got.isnan() & want.isnan()))
        assert not wrong.any(), (name, int(wrong.sum()), got[wrong][:4], want[wrong][:4])


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_finite(shape, dt):
    check_equal(integers(dt, *SHAPES[shape]))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("where", ["A", "B", "xt", "dyt"])
def test_one_operand(shape, dt, where):
    c = integers(dt, *SHAPES[shape])
    t = getattr(c, where)
    if t.dim() == 3:
        for a in range(t.shape[0]):
            t[a, 3, 5] = INF
            t[a, 1, t.shape[2] - 1] = -INF
    else:
        t[3, 0] = INF
        t[17, t.shape[1] // 2] = -INF
        t[5, t.shape[1] - 1] = INF
    want = definition(c)
    assert any((w.isinf()).any() for w in want)
    check_equal(c)


def classes(c):
    """Not finite where the definition is not, and of its sign."""
    for name, got, want in zip(NAMES, results(c), definition(c)):
        got = got.cpu()
        for kind in (torch.isnan, torch.isposinf, torch.isneginf):
            assert torch.equal(kind(got), kind(want)), (name, kind)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_values_that_split(shape, dt):
    """u and du have both parts, in f16 of either sign."""
    c = ref.Case(dt, *SHAPES[shape], 24, 40)
    c.B[:, 7, 2] = INF
    c.B[:, 9, 0] = -INF
    c.A[:, 4, 11] = INF
    classes(c)


@pytest.mark.parametrize("shape", ["one-token", "decode", "decode-33-ranks", "prompts",
                                   "prompts-24-ranks", "prompts-100-ranks"])
def test_f16_infinite_rank_beside_large_ones(shape):
    """An infinite u beside finite ones outside f16's range, which keep their
    sign and size: the scale is that of the finite ones."""
    c = integers("f16", *SHAPES[shape])
    c.xt.fill_(300.0)
    c.A.fill_(200.0)  # u about 1.4e6
    c.A[:, 3, 5] = INF
    c.B.fill_(-1.0)
    c.B[:, :, 3] = 1.0
    want = S.low_rank_add(c.yt, *c.args())
    busy = torch.zeros(c.T, dtype=torch.bool, device="cuda")
    for t, _, _, _ in c.runs():
        busy[t] = True
    assert (want[:, busy] == INF).all() and torch.equal(want[:, ~busy], c.yt[:, ~busy])
    # du beside it: B's infinity in one rank, dx = A^T du with opposite signs
    c = integers("f16", *SHAPES[shape])
    c.dyt.fill_(300.0)
    c.B.fill_(200.0)
    c.B[:, 3, 2] = INF
    c.A.fill_(-1.0)
    c.A[:, 2] = 1.0
    dx, dA, _ = S.low_rank_backward(c.dyt, *c.args())
    assert (dx[:, busy] == INF).all() and not dx[:, ~busy].any()
