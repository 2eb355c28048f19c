"""Low-rank adapters of many requests on the GPU against the float64 reference
(lowrank_ref), each value within the bound that its roundings allow."""
import pytest
import torch

import unstructured_sparse_linear_amd as S
import lowrank_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "f16", "bf16"]

# requests' lengths, adapters, pool, rank, features in and out
SHAPES = {
    "one-token": dict(lengths=[1], adapter=[2], n=3, R=16, n_in=256, n_out=320),
    "one-token-odd": dict(lengths=[1], adapter=[0], n=1, R=1, n_in=257, n_out=33),
    "tiny-features": dict(lengths=[2, 3], adapter=[0, 1], n=2, R=2, n_in=3, n_out=2),
    "decode": dict(lengths=[1] * 64, adapter=[(7 * i) % 9 - 1 for i in range(64)], n=8, R=16,
                   n_in=512, n_out=416),
    "decode-33": dict(lengths=[1] * 33, adapter=[i % 33 for i in range(33)], n=33, R=17,
                      n_in=300, n_out=129),
    "decode-200": dict(lengths=[1] * 200, adapter=[i % 11 for i in range(200)], n=11, R=8,
                       n_in=128, n_out=96),
    "prompts": dict(lengths=[100, 37, 1, 300, 74], adapter=[1, 0, 2, -1, 1], n=3, R=32, n_in=384,
                    n_out=512),
    "prompts-odd": dict(lengths=[131, 1, 250, 77], adapter=[0, 2, 1, 0], n=3, R=24, n_in=333,
                        n_out=271),
    "long": dict(lengths=[1200, 803], adapter=[0, 1], n=2, R=64, n_in=1000, n_out=1032),
    "empty-requests": dict(lengths=[0, 40, 0, 0, 25, 0], adapter=[1, 0, 1, 0, 1, 0], n=2, R=4,
                           n_in=96, n_out=64),
    "holes": dict(lengths=[30, 50], adapter=[0, 1], n=2, R=16, n_in=160, n_out=144, lead=21,
                  tail=70),
    "outside-pool": dict(lengths=[9, 9, 9, 9], adapter=[-1, 5, 1, -2 ** 31], n=2, R=8, n_in=64,
                         n_out=64),
    "ragged-ranks": dict(lengths=[50, 60, 70, 80], adapter=[0, 1, 2, 3], n=4, R=32, n_in=256,
                         n_out=208, ranks=[0, 1, 17, 40]),
    "rank-33": dict(lengths=[65], adapter=[0], n=1, R=33, n_in=128, n_out=160),
    "rank-100": dict(lengths=[64, 30], adapter=[1, 0], n=2, R=100, n_in=256, n_out=256,
                     ranks=[100, 71]),
    "rank-256": dict(lengths=[90], adapter=[0], n=1, R=256, n_in=320, n_out=288),
    "rows-apart": dict(lengths=[33, 48], adapter=[0, 1], n=2, R=16, n_in=200, n_out=120, pad=3),
    "no-scale": dict(lengths=[17], adapter=[0], n=1, R=16, n_in=64, n_out=64, scaled=False),
}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    S.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_add(shape, dt):
    c = ref.Case(dt, **SHAPES[shape])
    want = ref.add(c)
    got = S.low_rank_add(c.yt, *c.args())
    ref.check(got, want, "add")
    assert torch.equal(got, S.low_rank_add(c.yt, *c.args()))
    # in place, and tokens without an adapter keep their bits
    y = c.yt.clone(memory_format=torch.preserve_format)
    assert S.low_rank_add(y, *c.args(), out=y) is y
    assert torch.equal(y, got)
    idle = torch.ones(c.T, dtype=torch.bool, device="cuda")
    for t, _, _, _ in c.runs():
        idle[t] = False
    assert torch.equal(got[:, idle], c.yt[:, idle])


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_project(shape, dt):
    c = ref.Case(dt, **SHAPES[shape])
    got = S.low_rank_project(c.W, *c.args())
    ref.check(got, ref.project(c), "project")
    assert torch.equal(got, S.low_rank_project(c.W, *c.args()))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dt):
    c = ref.Case(dt, **SHAPES[shape])
    got = S.low_rank_backward(c.dyt, *c.args())
    for name, g, w in zip(("dx", "dA", "dB"), got, ref.backward(c)):
        ref.check(g, w, name)
    for g, h in zip(got, S.low_rank_backward(c.dyt, *c.args())):
        assert torch.equal(g, h)


@pytest.mark.parametrize("T", [0, 7])
def test_nothing_to_do(T):
    """No tokens, and tokens without a request."""
    kw = dict(lengths=[], adapter=[], n=2, R=4, n_in=32, n_out=48, lead=T)
    c = ref.Case("bf16", **kw)
    assert torch.equal(S.low_rank_add(c.yt, *c.args()), c.yt)
    ref.check(S.low_rank_project(c.W, *c.args()), ref.project(c))
    dx, dA, dB = S.low_rank_backward(c.dyt, *c.args())
    assert dx.shape == (32, T) and not dx.any() and not dA.any() and not dB.any()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("lengths", [[1] * 20, [40, 3, 90]])
def test_a_request_keeps_its_infinities(dt, lengths):
    """NaN and infinity in one request's tokens, in an unused adapter and past
    an adapter's rank leave every other result as it is."""
    S_ = len(lengths)
    c = ref.Case(dt, lengths, [i % 3 for i in range(S_)], 4, 20, 160, 144, ranks=[20, 7, 13, 20])
    clean = [S.low_rank_add(c.yt, *c.args()), S.low_rank_project(c.W, *c.args()),
             *S.low_rank_backward(c.dyt, *c.args())]
    bad = next(i for i in range(S_) if c.ad[i] == 1)
    other = torch.ones(c.T, dtype=torch.bool, device="cuda")
    for i in range(S_):
        if c.ad[i] == 1:
            other[c.off[i]:c.off[i + 1]] = False
    hurt = slice(c.off[bad], c.off[bad + 1])
    c.xt[5, hurt] = float("nan")
    c.xt[6, hurt] = float("inf")
    c.dyt[3, hurt] = float("-inf")
    c.A[3] = float("nan")
    c.B[3] = float("inf")
    for a, k in enumerate(c.rk):
        c.A[a, k:] = float("nan")
        c.B[a, :, k:] = float("inf")
    got = [S.low_rank_add(c.yt, *c.args()), S.low_rank_project(c.W, *c.args()),
           *S.low_rank_backward(c.dyt, *c.args())]
    for g, w in zip(got[:3], clean[:3]):
        assert torch.equal(g[:, other], w[:, other])
    for g, w in zip(got[3:], clean[3:]):
        for a in (0, 2, 3):
            assert torch.equal(g[a], w[a])
    assert not torch.isfinite(got[0][:, hurt]).any()
    assert not torch.isfinite(got[3][1, :7, 5]).any()
    assert not got[3][1, 7:].any() and not got[4][1, :, 7:].any()


@pytest.mark.parametrize("a,b,x", [(1e-3, 1e3, 1e-3), (3e4, 1e-3, 1.0)])
def test_f16_ranges(a, b, x):
    """u far outside f16's range, brought back by B: u is held in fp32."""
    c = ref.Case("f16", [70, 1, 30], [0, 1, 0], 2, 16, 512, 96)
    c.A.mul_(a)
    c.B.mul_(b)
    c.xt.mul_(x)
    c.yt.mul_(1e-3)
    c.dyt.mul_(1e-3)
    ref.check(S.low_rank_add(c.yt, *c.args()), ref.add(c), "add")
    ref.check(S.low_rank_project(c.W, *c.args()), ref.project(c), "project")
    for name, g, w in zip(("dx", "dA", "dB"), S.low_rank_backward(c.dyt, *c.args()),
                          ref.backward(c)):
        ref.check(g, w, name)


def test_offsets_that_do_not_ascend_stay_in_bounds():
    """Unspecified adapters, but every access in bounds and other calls unharmed."""
    c = ref.Case("bf16", [40, 30, 30], [0, 1, 0], 2, 16, 128, 128)
    for off in ([90, 10, 200, 5], [-50, 300, -1, 100], [2 ** 31 - 1, -2 ** 31, 50, 60]):
        args = (c.xt, c.A, c.B, torch.tensor(off, dtype=torch.int32, device="cuda"), c.adapter,
                c.scale, c.ranks)
        assert S.low_rank_add(c.yt, *args).shape == c.yt.shape
        assert S.low_rank_project(c.W, *args).shape == c.yt.shape
        S.low_rank_backward(c.dyt, *args)
    torch.cuda.synchronize()
    ref.check(S.low_rank_add(c.yt, *c.args()), ref.add(c), "add")


def test_positions_past_32_bits():
    """y and dx of more than 2^31 values, rows of odd length."""
    T, n_in, n_out = 262_147, 8200, 8200
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    xt, yt = normal(n_in, T), normal(n_out, T)
    assert yt.numel() > 2 ** 31
    A, B = normal(1, 4, n_in) * 0.01, normal(1, n_out, 4)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    ad = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = S.low_rank_add(yt, xt, A, B, off, ad)
    dx, dA, dB = S.low_rank_backward(yt, xt, A, B, off, ad)
    at = torch.tensor([0, 1, 77_777, T - 2, T - 1], device="cuda")
    x, y = xt[:, at].double(), yt[:, at].double()
    A, B = A[0].double(), B[0].double()
    eps = 2.0 ** -8
    for g_, want, mag in (
            (got[:, at], y + ref.mm(B, ref.mm(A, x)),
             y.abs() + B.abs().sum(1, keepdim=True) * ref.mm(A.abs(), x.abs()).amax(0)),
            (dx[:, at], ref.mm(A.t(), ref.mm(B.t(), y)),
             A.abs().sum(0)[:, None] * ref.mm(B.t().abs(), y.abs()).amax(0))):
        rel = ref.sum_error(n_in, 4) + ref.SPLIT["bf16"]
        assert ((g_.double() - want).abs() <= eps * want.abs() * (1 + 2 * rel) + rel * mag).all()
    # the gradients' last rows, in float64 over blocks of tokens
    row = torch.zeros(4, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(row)
    for t in range(0, T, 65536):
        x, y = xt[:, t:t + 65536].double(), yt[-1, t:t + 65536].double()
        row += ref.mm(ref.mm(A, x), y[:, None])[:, 0]
        mag += y.abs().sum() * ref.mm(A.abs(), x.abs()).amax(1)
    rel = ref.sum_error(n_in, T) + ref.SPLIT["bf16"]
    assert ((dB[0, -1].double() - row).abs() <= eps * row.abs() * (1 + 2 * rel) + rel * mag).all()


def test_gradients_against_differences():
    """<dL/dtheta, d> against (L(theta + h d) - L(theta - h d)) / 2h in f32: y is
    bilinear in (A, B), so the difference in one of them has no third-order
    term; what is left is fp32 rounding of y, 2^-24 (in + R + 8) of its terms'
    magnitude a value, over h."""
    c = ref.Case("f32", [50, 13, 90], [1, 0, 1], 2, 8, 96, 80)
    dx, dA, dB = S.low_rank_backward(c.dyt, *c.args())
    g = torch.Generator(device="cuda").manual_seed(3)
    _, bound = ref.add(c)
    noise = (bound * c.dyt.abs().double()).sum().item()
    h = 0.5
    for name, grad in (("xt", dx), ("A", dA), ("B", dB)):
        at = getattr(c, name)
        d = torch.randn(at.shape, generator=g, device="cuda").sign()  # +-h: exact enough steps
        side = []
        for s in (h, -h):
            setattr(c, name, at + s * d)
            _, b = ref.add(c)
            noise = max(noise, (b * c.dyt.abs().double()).sum().item())
            side.append((S.low_rank_add(c.yt, *c.args()).double() * c.dyt.double()).sum().item())
        setattr(c, name, at)
        slope = (side[0] - side[1]) / (2 * h)
        want = (grad.double() * d.double()).sum().item()
        # the steps at +- s d round once in fp32, as does the gradient
        slack = 2 * noise / (2 * h) + 2.0 ** -22 * (grad.double().abs() * (at.double().abs() / h + 1)).sum().item()
        own = dict(zip(("xt", "A", "B"), ref.backward(c)))[name][1].sum().item()
        assert abs(slope - want) <= slack + own, (name, slope, want)


def test_module_trains_like_autograd_of_the_formula():
    c = ref.Case("f32", [60, 21, 47], [0, -1, 2], 3, 16, 128, 112, ranks=[16, 4, 9])
    m = S.LowRankAdapters(3, 16, 128, 112, scale=c.scale, ranks=c.ranks)
    assert torch.equal(m(c.yt, c.xt, c.offsets, c.adapter), c.yt)  # B starts at zero
    with torch.no_grad():
        m.A.copy_(c.A)
        m.B.copy_(c.B)
    x, y = c.xt.clone().requires_grad_(), c.yt.clone().requires_grad_()
    m(y, x, c.offsets, c.adapter).backward(c.dyt)
    for g, w in zip((x.grad, m.A.grad, m.B.grad), ref.backward(c)):
        ref.check(g, w)
    assert torch.equal(y.grad, c.dyt)
    ref.check(m.project(c.W, c.xt, c.offsets, c.adapter), ref.project(c))


def test_calls_on_another_stream():
    c = ref.Case("bf16", [100, 29], [0, 1], 2, 16, 256, 256)
    want = ref.add(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs = [S.low_rank_add(c.yt, *c.args()) for _ in range(8)]
        grads = S.low_rank_backward(c.dyt, *c.args())
    other = [S.low_rank_add(c.yt, *c.args()) for _ in range(8)]
    torch.cuda.current_stream().wait_stream(s)
    for o in outs + other:
        ref.check(o, want)
        assert torch.equal(o, outs[0])
    for g, w in zip(grads, ref.backward(c)):
        ref.check(g, w)


def test_captured_calls_replay():
    """A training step's calls in a graph, replayed on new inputs with eager
    work between the replays."""
    cases = [ref.Case("f16", [60, 5, 130], [i % 2, 1, 0], 2, 32, 320, 288, seed=i)
             for i in range(4)]
    c = cases[0]
    names = ("xt", "yt", "dyt", "W", "A", "B", "scale", "adapter")

    def step():
        y = S.low_rank_add(c.yt, *c.args())
        p = S.low_rank_project(c.W, *c.args())
        dx, dA, dB = S.low_rank_backward(c.dyt, *c.args())
        return y, p, dx, dA, dB

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in (1, 2, 3, 1):
        for name in names:
            getattr(c, name).copy_(getattr(cases[k], name))
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        for o, e in zip(outs, eager):
            assert torch.equal(o, e)
