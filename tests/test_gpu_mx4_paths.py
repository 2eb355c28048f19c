"""Every tile shape and cut of the 4-bit products, offsets past 32 bits, rows far apart,
two streams at once, and a captured training step."""
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


def whole_matrix(seed, rows, cols, low=128, high=129):
    codes, scales = ref.random_mx4(np.random.default_rng(seed), rows, cols, low, high)
    W = S.Mx4Matrix(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), cols)
    return W, S.mx4_dequantize(W).double()


def whole_numbers(shape, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device="cuda").to(ref.DTYPES[dtype])


# rows, cols, tokens, transposed: large tiles whole, large with a few past a round of
# 256, small in pieces, small whole; odd sizes at every end
TILES = [(4097, 130, 2011, False), (4097, 530, 2011, False), (2049, 1090, 257, False),
         (1030, 4100, 190, False), (4096, 70, 1100, False), (130, 4097, 2100, True),
         (530, 4352, 4090, True), (1090, 2049, 257, True), (4100, 300, 190, True),
         (70, 4100, 1100, True)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,tokens,transposed", TILES)
def test_tiles(dtype, rows, cols, tokens, transposed):
    """Whole numbers: sums that f32 holds exactly, rounded once."""
    W, w = whole_matrix([rows, cols], rows, cols)
    m = w.t().contiguous() if transposed else w
    # beside x lie NaN, as in a padded batch
    big = torch.full((m.shape[1], tokens + 3), float("nan"), dtype=ref.DTYPES[dtype], device="cuda")
    x = big[:, 1:tokens + 1]
    x.copy_(whole_numbers((m.shape[1], tokens), dtype))
    want = torch.mm(m, x.double())
    assert float(want.abs().max()) < 2 ** 24
    out = torch.full((m.shape[0] + 1, tokens + 5), 7.0, dtype=x.dtype, device="cuda")
    S.mx4_matmul(W, x, transposed=transposed, out=out[:-1, 2:tokens + 2])
    assert torch.equal(out[:-1, 2:tokens + 2], want.to(x.dtype))
    assert (out[-1] == 7).all() and (out[:, :2] == 7).all() and (out[:, tokens + 2:] == 7).all()


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows,cols,tokens", [(2100, 300, 2100), (300, 2100, 2100), (200, 520, 150),
                                              (520, 200, 150)])
@pytest.mark.parametrize("scale", [0, 90, 103, 141, 150])
def test_one_wide_block_in_f16(rows, cols, tokens, transposed, scale):
    """One block whose scale f16 does not hold, among others: its tile runs on bf16, and
    nothing is lost."""
    W, _ = whole_matrix(scale, rows, cols, low=118, high=121)
    W.scales[rows - 2, (cols // 32) // 2] = scale
    w = S.mx4_dequantize(W).double()
    m = w.t().contiguous() if transposed else w
    x = whole_numbers((m.shape[1], tokens), "f16", scale)
    want, size = torch.mm(m, x.double()), torch.mm(m.abs(), x.double().abs())
    got = S.mx4_matmul(W, x, transposed=transposed).double()
    limit = torch.from_numpy(ref.bound(want.cpu().numpy(), m.shape[1], size.cpu().numpy(), "f16"))
    limit = limit.cuda()
    # from 65520 on a value rounds to an infinity
    fine = (got - want).abs() <= limit
    assert (fine | (torch.isinf(got) & (want.abs() + limit >= 65520))).all()
    must = want.abs() - limit >= 65520
    assert torch.isinf(got[must]).all()


@pytest.mark.parametrize("tokens", [4090, 3900])
def test_wide_blocks_in_large_tiles(tokens):
    """Every tile of 256 square, whole and in pieces, makes its tokens in two halves, one
    after the other in the same shared memory; the last half may lie past the tokens."""
    rows, cols = 530, 4352
    W, _ = whole_matrix(4, rows, cols, low=118, high=121)
    W.scales[::128, ::4] = 90
    w = S.mx4_dequantize(W).double().t().contiguous()
    x = whole_numbers((rows, tokens), "f16", 4)
    want, size = torch.mm(w, x.double()), torch.mm(w.abs(), x.double().abs())
    limit = torch.from_numpy(ref.bound(want.cpu().numpy(), rows, size.cpu().numpy(), "f16")).cuda()
    got = [S.mx4_matmul(W, x, transposed=True) for _ in range(3)]
    assert ((got[0].double() - want).abs() <= limit).all()
    assert torch.equal(got[1], got[0]) and torch.equal(got[2], got[0])


# tiles of 256, 128 and 64 square, in pieces or whole
FOUR = [(2570, 300, 4090), (2049, 290, 2049), (2050, 1000, 300), (300, 4097, 70), (70, 8200, 33)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,tokens", FOUR)
def test_tiles_of_two(dtype, rows, cols, tokens):
    W, w = whole_matrix([rows, 1], rows, cols)
    X, x = whole_matrix([tokens, 2], tokens, cols, low=128, high=128)
    want = torch.mm(w, x.t().contiguous())
    assert float(want.abs().max()) < 2 ** 24
    out = torch.full((rows + 1, tokens + 5), 7.0, dtype=ref.DTYPES[dtype], device="cuda")
    S.mx4_matmul(W, X, out=out[:-1, 2:tokens + 2])
    assert torch.equal(out[:-1, 2:tokens + 2], want.to(ref.DTYPES[dtype]))
    assert (out[-1] == 7).all() and (out[:, :2] == 7).all() and (out[:, tokens + 2:] == 7).all()
    assert torch.equal(S.mx4_matmul(W, X, out_dtype=ref.DTYPES[dtype]), out[:-1, 2:tokens + 2])


def test_matrix_by_itself():
    W, w = whole_matrix(3, 200, 300)
    assert torch.equal(S.mx4_matmul(W, W).double(), torch.mm(w, w.t().contiguous()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 5, 150])
@pytest.mark.parametrize("lead", [(1 << 21) + 7, (1 << 24) + 5])
def test_rows_far_apart(dtype, tokens, lead):
    """Rows of x and of the output further apart than 32 bits count."""
    cols = (1 << 32) // lead // 2 + 40
    W, w = whole_matrix(lead, 70, cols)
    big = torch.empty(cols, lead, dtype=ref.DTYPES[dtype], device="cuda")
    x = big[:, lead - tokens - 1:lead - 1]
    x.copy_(whole_numbers((cols, tokens), dtype))
    want = torch.mm(w, x.double()).to(x.dtype)
    assert torch.equal(S.mx4_matmul(W, x), want)
    x = big[:70, 3:tokens + 3]
    x.copy_(whole_numbers((70, tokens), dtype))
    out = big[:, lead - tokens - 1:lead - 1]
    S.mx4_matmul(W, x, transposed=True, out=out)
    assert torch.equal(out, torch.mm(w.t().contiguous(), x.double()).to(x.dtype))
    del big, x, out
    torch.cuda.empty_cache()


def test_matrix_of_more_than_32_bits():
    """Quantisation, dequantisation and one token's product past 4 GiB of codes, and past
    what one launch takes (2^31 words of eight elements)."""
    rows, cols = (1 << 19) + 300, 32800
    assert rows * 4 * 1025 > 1 << 31
    w = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    ends = [slice(0, 40), slice(rows - 40, rows)]
    g = torch.Generator(device="cuda").manual_seed(1)
    for e in ends:
        w[e] = torch.randn(40, cols, generator=g, device="cuda").bfloat16()
    W = S.mx4_quantize(w)
    x = whole_numbers((cols, 1), "bf16")
    y = S.mx4_matmul(W, x)
    for e in ends:
        small = S.mx4_quantize(w[e])
        assert torch.equal(W.codes[e], small.codes) and torch.equal(W.scales[e], small.scales)
        assert torch.equal(y[e], S.mx4_matmul(small, x))
    assert (W.scales[40:-40] == 127).all() and (y[40:-40] == 0).all()
    S.mx4_dequantize(W, torch.bfloat16, out=w)
    for e in ends:
        part = S.Mx4Matrix(W.codes[e], W.scales[e], cols)
        assert torch.equal(w[e], S.mx4_dequantize(part, torch.bfloat16))
    del w, W
    torch.cuda.empty_cache()


def test_two_streams_at_once():
    """Calls in flight together have workspaces of their own."""
    W, w = whole_matrix(5, 1000, 4100)
    xs = [whole_numbers((4100, 130), "bf16", i) for i in range(2)]
    want = [torch.mm(w, x.double()).bfloat16() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(S.mx4_matmul(W, xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_inference_mode():
    W, w = whole_matrix(6, 100, 70)
    with torch.inference_mode():
        x = whole_numbers((70, 9), "f32")
        assert torch.equal(S.mx4_linear(W, x), torch.mm(w, x.double()).float())
        assert torch.equal(S.dropout(x, 0.0, 1), x)


def test_captured_training_step():
    """Forward and backward of a frozen 4-bit layer with adapters and dropout in a graph:
    every replay draws its own masks and equals the eager step of the same state."""
    g = torch.Generator(device="cuda").manual_seed(2)
    base = S.Mx4Linear(torch.randn(200, 300, generator=g, device="cuda") * 300 ** -0.5)
    adapters = S.LowRankAdapters(2, 8, 300, 200, dropout=0.3, seed=11)
    with torch.no_grad():
        adapters.B.normal_(generator=g)
    xt = torch.zeros(300, 77, device="cuda", requires_grad=True)
    dy = torch.zeros(200, 77, device="cuda")
    off = torch.tensor([0, 30, 77], dtype=torch.int32, device="cuda")
    which = torch.tensor([1, 0], dtype=torch.int32, device="cuda")

    def step():
        y = adapters(base(xt), xt, off, which)
        return [y.detach(), *torch.autograd.grad(y, (xt, adapters.A, adapters.B), dy)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    seen = []
    for i in range(4):
        with torch.no_grad():
            xt.copy_(torch.randn(300, 77, generator=g, device="cuda"))
            dy.copy_(torch.randn(200, 77, generator=g, device="cuda"))
        before = adapters.dropout_state.clone()
        graph.replay()
        torch.cuda.synchronize()
        after = adapters.dropout_state.clone()
        assert (after - before).tolist() == [0, 1]
        result = [t.clone() for t in got]
        adapters.dropout_state.copy_(before)
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(result, want)), i
        seen.append(result[0])
    assert not torch.equal(seen[0], seen[1])


def test_a_state_that_moved_is_refused():
    """Adapters whose state moves on keep the masks of their own step: two forwards, then
    two backwards."""
    g = torch.Generator(device="cuda").manual_seed(3)
    adapters = S.LowRankAdapters(1, 4, 60, 50, dropout=0.5, seed=1)
    with torch.no_grad():
        adapters.B.normal_(generator=g)
    xt = torch.randn(60, 20, generator=g, device="cuda", requires_grad=True)
    off = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    which = torch.zeros(1, dtype=torch.int32, device="cuda")
    yt = torch.zeros(50, 20, device="cuda")
    ys = [adapters(yt, xt, off, which) for _ in range(2)]
    grads = [torch.autograd.grad(y.sum(), xt)[0] for y in ys]
    for step, grad in enumerate(grads):
        keep = torch.from_numpy(ref.dropout(np.ones((60, 20)), 0.5, 1, step)).cuda()
        A, B = adapters.A.detach().double(), adapters.B.detach().double()
        want = keep * (A[0].t() @ B[0].sum(0))[:, None]
        assert float((grad.double() - want).abs().max()) < 1e-5 * float(want.detach().abs().max())


def test_example():
    """The example runs, and its parts give what the calls give."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import four_bit_finetune as example
    losses, base, layer = example.finetune(steps=3, features=128, tokens=33)
    assert len(losses) == 3 and all(np.isfinite(losses))
    step, whole, four = example.serve(base, layer)
    assert step.shape == (128, 5) and whole.shape == four.shape == (128, 40)
    w = S.mx4_dequantize(base.weight).double().cpu().numpy()
    g = torch.Generator(device="cuda").manual_seed(1)
    xt = torch.randn(128, 5, generator=g, device="cuda").double().cpu().numpy()
    want = w @ xt
    A, B = (p.detach().double().cpu().numpy() for p in (layer.A, layer.B))
    for t in range(5):
        want[:, t] += B[t % 3] @ (A[t % 3] @ xt[:, t])
    assert np.abs(step.double().cpu().numpy() - want).max() < 1e-5 * np.abs(want).max()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1919, 300), (1921, 300), (2301, 33), (4100, 1000)])
def test_quantising_along_columns(dtype, rows, cols):
    """Few and many tiles of rows, each in its own order: the same bits as along the rows."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    big = torch.randn(cols, rows + 1, generator=g, device="cuda").to(ref.DTYPES[dtype])
    x = big[:, 1:].t()
    got, want = S.mx4_quantize(x), S.mx4_quantize(x.contiguous())
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
