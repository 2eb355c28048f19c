"""4-bit microscaled matrices against float64: the format, the products with dense
and with 4-bit activations, and the gradient."""
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


def matrix(rng, rows, cols, **kw):
    codes, scales = ref.random_mx4(rng, rows, cols, **kw)
    return (S.Mx4Matrix(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), cols),
            ref.dequantize(codes, scales, cols))


def rounded(x, dtype):
    """A float64 array in a type: the device tensor and the values it holds."""
    t = torch.from_numpy(x).to(ref.DTYPES[dtype])
    return t.cuda(), t.double().numpy()


def f64(t):
    return t.double().cpu().numpy()


def check(got, want, terms, magnitude, dtype, what=""):
    assert got.dtype == ref.DTYPES[dtype]
    g = f64(got)
    assert g.shape == want.shape
    with np.errstate(over="ignore"):
        limit = ref.bound(want, terms, magnitude, dtype)
    bad = ~(np.abs(g - want) <= limit)
    if dtype == "f16":
        # 65504 is the largest value; what rounds to 65536, from 65520 on, is an infinity
        may = np.abs(want) + limit >= 65520
        must = np.abs(want) - limit >= 65520
        bad = np.where(np.isinf(g), ~may | (np.sign(g) != np.sign(want)), bad | must)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.abs(g - want).max()))


SHAPES = [(1, 1), (3, 31), (5, 32), (2, 33), (70, 257), (64, 1024), (1, 4096), (129, 100)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("turned", [False, True])
def test_quantize(dtype, rows, cols, turned):
    rng = np.random.default_rng([rows, cols])
    x, v = rounded(rng.normal(size=(rows, cols)) * np.exp2(rng.integers(-9, 6, (rows, 1))), dtype)
    codes, scales = ref.quantize(v)
    w = x.t().contiguous().t() if turned else x
    Q = S.mx4_quantize(w)
    assert Q.shape == (rows, cols)
    assert np.array_equal(Q.scales.cpu().numpy(), scales)
    assert np.array_equal(Q.codes.cpu().numpy(), codes)
    for t in ref.DTYPES.values():
        assert np.array_equal(f64(S.mx4_dequantize(Q, t)), ref.dequantize(codes, scales, cols))


@pytest.mark.parametrize("turned", [False, True])
def test_quantize_strides(turned):
    """Rows or columns inside a larger matrix, at odd addresses."""
    rng = np.random.default_rng(5)
    for dtype in ref.DTYPES:
        x, v = rounded(rng.normal(size=(90, 131)), dtype)
        w, want = x[3:70, 1:100], v[3:70, 1:100]
        if turned:
            w, want = w.t(), want.T
        codes, scales = ref.quantize(want)
        Q = S.mx4_quantize(w)
        assert np.array_equal(Q.codes.cpu().numpy(), codes)
        assert np.array_equal(Q.scales.cpu().numpy(), scales)


@pytest.mark.parametrize("turned", [False, True])
def test_quantize_extremes(turned):
    """Ties, saturation, zeros, subnormals, infinities and NaN, blocks apart."""
    w = np.zeros((16, 96), np.float32)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.99, 0.2500001, 0.7499999])
    w[0, :11] = ties
    w[1, :11] = -ties
    w[2, 0], w[2, 40] = np.inf, 1.0
    w[3, 95], w[3, 40] = np.nan, 1.0
    w[4, 3] = -np.inf
    w[5, :32] = 2.0 ** -130 * np.arange(32)
    w[6, :32] = 2.0 ** -149
    w[7, :3] = [3.4e38, -3e38, 1e38]
    w[8, :2] = [2.0 ** -127, -2.0 ** -128]
    w[9, 32:64] = -0.0
    w[10, 0] = np.nextafter(np.float32(8), np.float32(0))
    w[11, 0] = 2.0 ** -125
    w[12, 0] = 2.0 ** -126 * 1.99
    codes, scales = ref.quantize(w.astype(np.float64))
    x = torch.from_numpy(w).cuda()
    Q = S.mx4_quantize(x.t().contiguous().t() if turned else x)
    assert np.array_equal(Q.scales.cpu().numpy(), scales)
    assert np.array_equal(Q.codes.cpu().numpy(), codes)
    want = ref.dequantize(codes, scales, 96)
    assert np.array_equal(f64(S.mx4_dequantize(Q)), want, equal_nan=True)
    # f16 cannot hold all of them: the nearest it can
    with np.errstate(over="ignore"):
        half = want.astype(np.float16).astype(np.float64)
    assert np.array_equal(f64(S.mx4_dequantize(Q, torch.float16)), half, equal_nan=True)


def test_dequantize_every_element_and_scale():
    i = np.tile(np.arange(16, dtype=np.uint8), 2)
    codes = np.repeat((i[0::2] | (i[1::2] << 4))[None], 256, 0)
    scales = np.arange(256, dtype=np.uint8)[:, None]
    W = S.Mx4Matrix(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 32)
    want = ref.dequantize(codes, scales, 32)
    with np.errstate(over="ignore"):
        f32 = want.astype(np.float32).astype(np.float64)
    assert np.array_equal(f64(S.mx4_dequantize(W)), f32, equal_nan=True)
    assert np.array_equal(f64(S.mx4_dequantize(W, torch.bfloat16)), f32, equal_nan=True)
    out = torch.full((256, 40), 7.0, device="cuda")
    assert S.mx4_dequantize(W, out=out[:, 3:35]) is not None
    assert np.array_equal(f64(out[:, 3:35]), f32, equal_nan=True)
    assert (out[:, :3] == 7).all() and (out[:, 35:] == 7).all()


# tokens from one to several tiles, inner sizes around blocks and steps of 64
PRODUCTS = [(1, 1, 1), (5, 32, 1), (33, 31, 2), (64, 64, 3), (130, 200, 7), (100, 63, 8),
            (257, 65, 15), (96, 1024, 16), (40, 161, 17), (300, 520, 33), (128, 128, 64),
            (70, 96, 100), (513, 640, 129), (260, 1000, 255), (1030, 130, 257), (48, 2050, 300)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,tokens", PRODUCTS)
@pytest.mark.parametrize("transposed", [False, True])
def test_product(dtype, rows, cols, tokens, transposed):
    rng = np.random.default_rng([rows, cols, tokens])
    W, w = matrix(rng, rows, cols)
    m = w.T if transposed else w
    x, v = rounded(rng.normal(size=(m.shape[1], tokens)), dtype)
    got = S.mx4_matmul(W, x, transposed=transposed)
    check(got, m @ v, m.shape[1], np.abs(m) @ np.abs(v), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,tokens", PRODUCTS)
@pytest.mark.parametrize("transposed", [False, True])
def test_product_of_whole_numbers(dtype, rows, cols, tokens, transposed):
    """Sums that f32 holds exactly come out exactly, rounded once."""
    rng = np.random.default_rng([rows, cols, tokens, 1])
    W, w = matrix(rng, rows, cols, low=128, high=129)
    m = w.T if transposed else w
    x, v = rounded(rng.integers(-4, 5, (m.shape[1], tokens)).astype(np.float64), dtype)
    want = torch.from_numpy(m @ v)
    assert float(want.abs().max()) < 2 ** 24
    got = S.mx4_matmul(W, x, transposed=transposed)
    assert torch.equal(got.cpu(), want.to(ref.DTYPES[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 5, 31, 200])
@pytest.mark.parametrize("transposed", [False, True])
def test_product_strides_and_out(dtype, tokens, transposed):
    """x and out inside larger matrices whose other elements are NaN, or stay."""
    rng = np.random.default_rng(tokens)
    W, w = matrix(rng, 150, 200)
    m = w.T if transposed else w
    x, v = rounded(rng.normal(size=(m.shape[1], tokens)), dtype)
    for lead, trail in ((1, 0), (3, 5), (8, 24)):
        big = torch.full((m.shape[1] + 2, lead + tokens + trail), float("nan"),
                         dtype=x.dtype, device="cuda")
        inner = big[1:-1, lead:lead + tokens]
        inner.copy_(x)
        out = torch.full((m.shape[0] + 2, lead + tokens + trail), 7.0, dtype=x.dtype, device="cuda")
        to = out[1:-1, lead:lead + tokens]
        assert S.mx4_matmul(W, inner, transposed=transposed, out=to) is to
        check(to, m @ v, m.shape[1], np.abs(m) @ np.abs(v), dtype)
        to.fill_(7.0)
        assert (out == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 20, 150])
@pytest.mark.parametrize("transposed", [False, True])
def test_product_wide_scales(dtype, tokens, transposed):
    """Scales far outside the range of f16 beside ordinary ones: nothing is lost."""
    rng = np.random.default_rng(tokens + 7)
    W, w = matrix(rng, 96, 160, low=60, high=150)
    m = w.T if transposed else w
    x, v = rounded(rng.normal(size=(m.shape[1], tokens)), dtype)
    want, size = m @ v, np.abs(m) @ np.abs(v)
    check(S.mx4_matmul(W, x, transposed=transposed), want, m.shape[1], size, dtype)
    # only the smallest scales: sums far below one
    W, w = matrix(rng, 96, 160, low=60, high=90)
    m = w.T if transposed else w
    x, v = rounded(rng.normal(size=(m.shape[1], tokens)) * 1000, dtype)
    check(S.mx4_matmul(W, x, transposed=transposed), m @ v, m.shape[1], np.abs(m) @ np.abs(v),
          dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 9, 140])
@pytest.mark.parametrize("transposed", [False, True])
def test_product_of_infinities_and_nan(dtype, tokens, transposed):
    """Only the outputs that an infinity or NaN belongs to are touched by it, as in the
    definition (zero times infinity is NaN)."""
    rng = np.random.default_rng(tokens + 70)
    codes, scales = ref.random_mx4(rng, 70, 100)
    scales[3, 1] = 255                                  # a NaN block of W
    W = S.Mx4Matrix(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 100)
    w = ref.dequantize(codes, scales, 100)
    m = w.T if transposed else w
    x, v = rounded(rng.normal(size=(m.shape[1], tokens)), dtype)
    v[7, 0], v[20, tokens // 2], v[33, tokens - 1] = np.inf, -np.inf, np.nan
    x[7, 0], x[20, tokens // 2], x[33, tokens - 1] = np.inf, -np.inf, np.nan
    with np.errstate(invalid="ignore"):
        want = np.stack([(m * v[:, t]).sum(1) for t in range(tokens)], 1)
    got = f64(S.mx4_matmul(W, x, transposed=transposed))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isinf(got), np.isinf(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    fine = np.isfinite(want)
    size = np.abs(np.nan_to_num(m)) @ np.abs(np.nan_to_num(v, posinf=0, neginf=0))
    limit = ref.bound(np.where(fine, want, 0), m.shape[1], size, dtype)
    assert (np.abs(got[fine] - want[fine]) <= limit[fine]).all()


def test_product_of_subnormal_weights_and_values():
    """f32 and bf16 values down to the smallest, and blocks of the smallest scales."""
    rng = np.random.default_rng(3)
    for dtype in ("f32", "bf16"):
        for low, high, std in ((0, 2, 2.0 ** 100), (128, 134, 2.0 ** -133)):
            W, w = matrix(rng, 40, 64, low=low, high=high)
            x, v = rounded(rng.normal(size=(64, 20)) * std, dtype)
            got, want, size = S.mx4_matmul(W, x), w @ v, np.abs(w) @ np.abs(v)
            # an f32 value is the sum of three bf16 parts, cut towards zero; what bf16 holds
            # are multiples of 2^-133, so up to that is left out of each value (of those
            # under 2^-109, whose last bit lies below) and, times w, of each product
            lost = 2.0 ** -133 * np.abs(w).sum(1, keepdims=True) if dtype == "f32" else 0.0
            limit = ref.bound(want, 64, size, dtype) + lost
            assert (np.abs(f64(got) - want) <= limit).all(), (dtype, low)


@pytest.mark.parametrize("transposed", [False, True])
def test_product_without_tokens(transposed):
    W, w = matrix(np.random.default_rng(0), 40, 70)
    m = w.T if transposed else w
    x = torch.empty(m.shape[1], 0, device="cuda")
    assert S.mx4_matmul(W, x, transposed=transposed).shape == (m.shape[0], 0)


FOUR = [(1, 1, 1), (33, 31, 2), (64, 64, 40), (130, 200, 7), (257, 129, 150), (300, 1000, 260),
        (128, 4096, 128), (513, 640, 129)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,tokens", FOUR)
def test_product_of_two(dtype, rows, cols, tokens):
    rng = np.random.default_rng([rows, cols, tokens, 2])
    W, w = matrix(rng, rows, cols)
    X, x = matrix(rng, tokens, cols, low=120, high=130)
    got = S.mx4_matmul(W, X, out_dtype=ref.DTYPES[dtype])
    check(got, w @ x.T, cols, np.abs(w) @ np.abs(x).T, dtype)
    big = torch.full((rows, tokens + 9), 7.0, dtype=ref.DTYPES[dtype], device="cuda")
    S.mx4_matmul(W, X, out=big[:, 4:tokens + 4])
    assert torch.equal(big[:, 4:tokens + 4], got)
    assert (big[:, :4] == 7).all() and (big[:, tokens + 4:] == 7).all()


@pytest.mark.parametrize("rows,cols,tokens", FOUR)
def test_product_of_two_of_whole_numbers(rows, cols, tokens):
    rng = np.random.default_rng([rows, cols, tokens, 3])
    W, w = matrix(rng, rows, cols, low=128, high=129)
    X, x = matrix(rng, tokens, cols, low=128, high=128)
    assert np.abs(w @ x.T).max() < 2 ** 24
    assert np.array_equal(f64(S.mx4_matmul(W, X)), w @ x.T)


def test_product_of_two_with_nan_and_extremes():
    rng = np.random.default_rng(11)
    codes, scales = ref.random_mx4(rng, 70, 100)
    scales[3, 1], scales[5, 3] = 255, 255
    W = S.Mx4Matrix(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 100)
    xcodes, xscales = ref.random_mx4(rng, 50, 100)
    xscales[40, 0] = 255
    X = S.Mx4Matrix(torch.from_numpy(xcodes).cuda(), torch.from_numpy(xscales).cuda(), 100)
    w, x = ref.dequantize(codes, scales, 100), ref.dequantize(xcodes, xscales, 100)
    nan = np.isnan(w).any(1)[:, None] | np.isnan(x).any(1)[None]
    got = f64(S.mx4_matmul(W, X))
    assert np.array_equal(np.isnan(got), nan)
    w, x = np.nan_to_num(w), np.nan_to_num(x)
    want, size = w @ x.T, np.abs(w) @ np.abs(x).T
    assert (np.abs(got - want) <= ref.bound(want, 100, size, "f32"))[~nan].all()


def test_quantized_activations():
    """mx4_quantize(xt.t()) and the product, as a prompt is served."""
    rng = np.random.default_rng(12)
    W, w = matrix(rng, 200, 300)
    x, v = rounded(rng.normal(size=(300, 77)), "bf16")
    X = S.mx4_quantize(x.t())
    xq = ref.dequantize(*ref.quantize(v.T), 300)
    got = S.mx4_matmul(W, X, out_dtype=torch.bfloat16)
    check(got, w @ xq.T, 300, np.abs(w) @ np.abs(xq).T, "bf16")


def test_linear_gradient():
    """The gradient against the formula and against differences, and the second one."""
    rng = np.random.default_rng(13)
    W, w = matrix(rng, 33, 70)
    x, v = rounded(rng.normal(size=(70, 9)), "f32")
    dy, d = rounded(rng.normal(size=(33, 9)), "f32")
    x.requires_grad_()
    y = S.mx4_linear(W, x)
    check(y.detach(), w @ v, 70, np.abs(w) @ np.abs(v), "f32")
    g, = torch.autograd.grad((y * dy).sum(), x)
    check(g, w.T @ d, 33, np.abs(w).T @ np.abs(d), "f32")
    # the loss is linear in x: a difference along e is the gradient along e
    e, ev = rounded(rng.integers(-2, 3, (70, 9)).astype(np.float64), "f32")
    diff = f64(S.mx4_linear(W, x.detach() + e) - y.detach()) * d
    slope = float((f64(g) * ev).sum())
    assert abs(diff.sum() - slope) < 1e-4 * (np.abs(w) @ np.abs(v) * np.abs(d)).sum()
    # through the square of the result: the second derivative is 2 W^T W
    y = S.mx4_linear(W, x)
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    h, = torch.autograd.grad((g * e).sum(), x)
    want = 2 * w.T @ (w @ ev)
    assert np.abs(f64(h) - want).max() < 1e-4 * np.abs(want).max()


def test_linear_module_and_adapters():
    """Adapters on a frozen 4-bit layer: training with dropout, then serving."""
    g = torch.Generator(device="cuda").manual_seed(0)
    weight = torch.randn(80, 96, generator=g, device="cuda") * 96 ** -0.5
    base = S.Mx4Linear(weight)
    W = f64(S.mx4_dequantize(base.weight))
    assert sorted(base.state_dict()) == ["codes", "scales"] and not list(base.parameters())
    adapters = S.LowRankAdapters(2, 8, 96, 80, dropout=0.25, seed=3)
    with torch.no_grad():
        adapters.B.normal_(generator=g)
    xt = torch.randn(96, 21, generator=g, device="cuda", requires_grad=True)
    off = torch.tensor([0, 13, 21], dtype=torch.int32, device="cuda")
    which = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    for step in range(2):
        assert adapters.dropout_state.tolist() == [3, step]
        y = adapters(base(xt), xt, off, which)
        dy = torch.randn(80, 21, generator=g, device="cuda")
        dx, dA = torch.autograd.grad(y, (xt, adapters.A), dy)
        x, d = f64(xt.detach()), f64(dy)
        keep = ref.dropout(np.ones((96, 21)), 0.25, 3, step)
        A, B = f64(adapters.A.detach()), f64(adapters.B.detach())
        want, wdx, wdA = W @ x, W.T @ d, np.zeros_like(A)
        for a, t in ((1, slice(0, 13)), (0, slice(13, 21))):
            want[:, t] += B[a] @ (A[a] @ (x * keep)[:, t])
            du = B[a].T @ d[:, t]
            wdx[:, t] += keep[:, t] * (A[a].T @ du)
            wdA[a] = du @ (x * keep)[:, t].T
        for got, w in ((y.detach(), want), (dx, wdx), (dA, wdA)):
            assert np.abs(f64(got) - w).max() < 1e-5 * np.abs(w).max()
    adapters.eval()
    with torch.no_grad():
        apart = adapters(base(xt), xt, off, which)
        together = adapters.project(base.weight, xt.detach(), off, which)
    assert adapters.dropout_state.tolist() == [3, 2]
    assert torch.equal(apart, together)


def test_other_stream_and_repeated_runs():
    """The same bits on another stream and in every run."""
    rng = np.random.default_rng(14)
    W, w = matrix(rng, 300, 520)
    x, _ = rounded(rng.normal(size=(520, 33)), "bf16")
    want = S.mx4_matmul(W, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [S.mx4_matmul(W, x) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_captured():
    """Quantisation, both products, the gradient and dropout in a graph, replayed with
    other inputs and eager work between."""
    rng = np.random.default_rng(15)
    W, _ = matrix(rng, 300, 520)
    x = torch.zeros(520, 33, dtype=torch.bfloat16, device="cuda")
    state = torch.zeros(2, dtype=torch.int64, device="cuda")

    def work():
        y = S.mx4_matmul(W, x)
        z = S.mx4_matmul(W, S.mx4_quantize(x.t()), out_dtype=torch.bfloat16)
        return y, z, S.mx4_matmul(W, y, transposed=True), S.dropout(x, 0.3, state)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for i in range(3):
        x.copy_(rounded(rng.normal(size=(520, 33)), "bf16")[0])
        state.copy_(torch.tensor([17, i]))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, work())), i
