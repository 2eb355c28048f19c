"""Dropout against the generator's definition: every element's bits, shapes, strides,
places past 32 bits, gradients and the device's seed."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import unstructured_sparse_linear_amd as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    S.lib()
    yield
    torch.cuda.synchronize()


SEED, STEP = 0x8badf00d12345678, 0x0123456789abcdef


def values(shape, dtype, seed=0):
    t = torch.from_numpy(np.random.default_rng(seed).normal(size=shape)).to(ref.DTYPES[dtype])
    return t.cuda(), t.double().numpy()


def expected(v, p, seed, step, dtype):
    """Kept values are multiplied in f32 and rounded once: equal bit for bit."""
    limit = int(np.floor(p * 65536 + 0.5))
    scale = np.float32(65536 / (65536 - limit)) if limit < 65536 else np.float32(0)
    keep = ref.random16(*v.shape, seed, step) >= limit
    with np.errstate(invalid="ignore"):
        y = np.where(keep, v.astype(np.float32) * scale, np.float32(0))
    return torch.from_numpy(y).to(ref.DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (3, 8), (5, 9), (70, 257), (300, 1), (2, 4096)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_every_element(dtype, shape, p):
    x, v = values(shape, dtype)
    got = S.dropout(x, p, SEED, STEP)
    assert torch.equal(got.cpu(), expected(v, p, SEED, STEP, dtype))
    state = torch.tensor([SEED - (1 << 64), STEP], dtype=torch.int64, device="cuda")
    assert torch.equal(S.dropout(x, p, state), got)
    assert torch.equal(S.dropout(x, p, SEED - (1 << 64), STEP), got)
    assert S.dropout(x, p, SEED, STEP, out=x) is x and torch.equal(x, got)


def test_smallest_and_largest_probabilities():
    x, v = values((64, 512), "f32")
    for p in (2.0 ** -17 - 1e-9, 2.0 ** -17, 2.0 ** -16, 1 - 2.0 ** -16, 1 - 2.0 ** -18):
        assert torch.equal(S.dropout(x, p, 5).cpu(), expected(v, p, 5, 0, "f32")), p


def test_shapes_and_strides():
    x, v = values((6, 10, 33), "bf16")
    want = expected(v.reshape(60, 33), 0.3, 9, 2, "bf16")
    assert torch.equal(S.dropout(x, 0.3, 9, 2).cpu(), want.reshape(6, 10, 33))
    flat, w = values((1000,), "f16")
    assert torch.equal(S.dropout(flat, 0.3, 9, 2).cpu(),
                       expected(w.reshape(1, -1), 0.3, 9, 2, "f16")[0])
    one, w = values((), "f32")
    assert torch.equal(S.dropout(one, 0.3, 9, 2).cpu(),
                       expected(w.reshape(1, 1), 0.3, 9, 2, "f32")[0, 0])
    for shape in ((0,), (0, 5), (5, 0), (2, 0, 3)):
        assert S.dropout(torch.empty(shape, device="cuda"), 0.3, 9).shape == shape
    # inside larger matrices, at odd addresses; what lies beside stays
    big, w = values((40, 101), "bf16")
    out = torch.full((40, 103), 7.0, dtype=torch.bfloat16, device="cuda")
    to = out[2:38, 5:96]
    assert S.dropout(big[3:39, 1:92], 0.3, 9, 2, out=to) is to
    assert torch.equal(to.cpu(), expected(w[3:39, 1:92], 0.3, 9, 2, "bf16"))
    to.fill_(7.0)
    assert (out == 7).all()


def test_dropped_places_hold_zero():
    x = torch.full((50, 300), float("nan"), device="cuda")
    x[:, ::2] = float("inf")
    keep = torch.from_numpy(ref.random16(50, 300, 1, 0) >= 32768)
    y = S.dropout(x, 0.5, 1).cpu()
    assert (y[~keep] == 0).all() and not torch.isfinite(y[keep]).any()


def test_gradient():
    """The same call on dy; against differences; a second derivative of zero."""
    x, v = values((30, 50), "f32")
    x.requires_grad_()
    dy, d = values((30, 50), "f32", 1)
    state = torch.tensor([4, 5], dtype=torch.int64, device="cuda")
    for seed in (4, state):
        y = S.dropout(x, 0.2, seed, 5)
        g, = torch.autograd.grad(y, x, dy, retain_graph=True)
        assert torch.equal(g, S.dropout(dy, 0.2, 4, 5))
        e = torch.zeros_like(x)
        e[11, 7], e[3, 40] = 1.0, -2.0
        slope = ((S.dropout(x.detach() + e, 0.2, 4, 5) - y.detach()).double() * dy.double()).sum()
        assert abs(float(slope - (g.double() * e.double()).sum())) < 1e-5
    # a transposed dy, and a graph of the gradient
    g, = torch.autograd.grad(S.dropout(x, 0.2, 4, 5), x, dy.t().contiguous().t())
    assert torch.equal(g, S.dropout(dy, 0.2, 4, 5))
    y = S.dropout(x, 0.2, 4, 5)
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    h, = torch.autograd.grad(g.sum(), x)
    keep = S.dropout(torch.ones_like(x), 0.2, 4, 5)
    assert torch.allclose(h, 2 * keep * keep, rtol=1e-6)
    # a state that moved on before the backward pass is refused
    y = S.dropout(x, 0.2, state)
    state[1].add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()


def test_mean_and_independence():
    """Rates of a large mask within five standard deviations, for rows, columns, steps
    and seeds apart."""
    n, p = 1 << 22, 0.1
    x = torch.ones(1 << 10, 1 << 12, device="cuda")
    dropped = {}
    for seed, step in ((1, 0), (1, 1), (2, 0), (1 << 40, 0)):
        dropped[seed, step] = S.dropout(x, p, seed, step) == 0
    sd = (n * p * (1 - p)) ** 0.5
    for d in dropped.values():
        assert abs(float(d.sum()) - n * (round(p * 65536) / 65536)) < 5 * sd
    both = (n * p * p * (1 - p * p)) ** 0.5
    base = dropped[1, 0]
    for other in list(dropped.values())[1:] + [base.roll(1, 0), base.roll(1, 1), base.roll(8, 1)]:
        assert abs(float((base & other).sum()) - n * p * p) < 5 * both


def test_rows_past_32_bits_of_elements():
    """A matrix of more than 2^32 elements, checked at its ends."""
    rows, cols = (1 << 21) + 5, 2056
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    S.dropout(x, 0.25, SEED, 3, out=x)
    for r in (0, (1 << 20) + 1, (1 << 31) // cols - 2, rows - 4):
        want = ref.random16(4, cols, SEED, 3, r) >= 16384
        assert np.array_equal((x[r:r + 4] != 0).cpu().numpy(), want)
    del x
    torch.cuda.empty_cache()


def test_more_than_one_launch():
    """More groups of eight columns than one launch takes: rows on both sides of the cut."""
    rows, cols = (1 << 21) + 5, 8200
    first = (1 << 31) // 1025
    assert first < rows - 8
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    S.dropout(x, 0.25, SEED, 4, out=x)
    for r in (0, first - 2, rows - 4):
        want = ref.random16(4, cols, SEED, 4, r) >= 16384
        assert np.array_equal((x[r:r + 4] != 0).cpu().numpy(), want)
    del x
    torch.cuda.empty_cache()


def test_every_element_once_over_launches():
    """In place, with rows whose groups do not fill the last workgroup of a launch: none of
    the next launch's elements is scaled twice."""
    cols = 24
    first = (1 << 31) // 3  # rows of the first launch
    rows = first + 200
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    S.dropout(x, 0.5, SEED, 5, out=x)
    want = torch.where(torch.from_numpy(ref.random16(200, cols, SEED, 5, first - 100) >= 32768),
                       2.0, 0.0)
    assert torch.equal(x[first - 100:first + 100].float().cpu(), want.float())
    del x
    torch.cuda.empty_cache()
