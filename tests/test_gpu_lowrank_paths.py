"""The low-rank adapter calls where a rule on sizes takes another kernel: a few
tokens with one adapter, several row tiles a workgroup, tiles of many adapters,
rows that start between two words; and the example that runs them together."""
import importlib.util
import os

import pytest
import torch

import unstructured_sparse_linear_amd as S
import lowrank_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "f16", "bf16"]

FEW = {  # up to 16 tokens, at most one adapter, up to 32 ranks: one launch
    "request-of-16": dict(lengths=[16], adapter=[2], n=3, R=16, n_in=515, n_out=300),
    "token-of-strided-x": dict(lengths=[1], adapter=[0], n=2, R=9, n_in=288, n_out=70, pad=3),
    "32-ranks": dict(lengths=[7], adapter=[1], n=2, R=32, n_in=640, n_out=272, ranks=[3, 29]),
    "one-adapter-of-many-requests": dict(lengths=[0] * 70 + [3, 0, 4, 1], adapter=[0] * 72 + [-1, 0],
                                         n=1, R=20, n_in=96, n_out=40, lead=2, tail=3),
    "no-adapter": dict(lengths=[5], adapter=[-1], n=2, R=8, n_in=64, n_out=33),
    "no-ranks": dict(lengths=[5], adapter=[1], n=2, R=8, n_in=64, n_out=33, ranks=[8, 0]),
    "five-features": dict(lengths=[3], adapter=[0], n=1, R=5, n_in=5, n_out=7),
    "long-features": dict(lengths=[1], adapter=[0], n=1, R=16, n_in=9000, n_out=48),
    "17-tokens": dict(lengths=[17], adapter=[0], n=1, R=16, n_in=160, n_out=96),
}
WIDE = {
    "two-row-tiles": dict(lengths=[1] * 20, adapter=[i % 6 - 1 for i in range(20)], n=5, R=16,
                          n_in=96, n_out=5003),
    "three-row-tiles": dict(lengths=[1] * 50, adapter=[i % 9 for i in range(50)], n=9, R=33,
                            n_in=70, n_out=9001, ranks=[33, 1, 0, 8, 9, 17, 32, 33, 16]),
    "three-row-tiles-200-ranks": dict(lengths=[30, 31], adapter=[0, 1], n=2, R=200, n_in=64,
                                      n_out=8300),
}
MANY = {
    "adapters-in-every-tile": dict(lengths=[(7 * i) % 23 for i in range(60)],
                                   adapter=[(11 * i) % 26 for i in range(60)], n=26, R=24,
                                   n_in=640, n_out=704),
    "192-tokens": dict(lengths=[192], adapter=[0], n=1, R=40, n_in=96, n_out=130),
    "193-tokens": dict(lengths=[193], adapter=[0], n=1, R=40, n_in=96, n_out=130),
    "256-requests": dict(lengths=[1] * 256, adapter=[i % 7 - 1 for i in range(256)], n=6, R=16,
                         n_in=160, n_out=100),
    "257-requests": dict(lengths=[1] * 257, adapter=[i % 7 - 1 for i in range(257)], n=6, R=16,
                         n_in=160, n_out=100),
    "64-ranks": dict(lengths=[(37 * i) % 90 + 1 for i in range(31)],
                     adapter=[(5 * i) % 8 - 1 for i in range(31)], n=7, R=64, n_in=321, n_out=384),
    "odd-rows": dict(lengths=[500, 1, 546], adapter=[0, 1, 0], n=2, R=32, n_in=200, n_out=216),
    "rows-between-words": dict(lengths=[100, 129], adapter=[0, 1], n=2, R=16, n_in=96, n_out=80,
                               pad=1),
    "256-ranks-of-many-adapters": dict(lengths=[(13 * i) % 40 for i in range(30)],
                                       adapter=[(7 * i) % 27 for i in range(30)], n=27, R=256,
                                       n_in=640, n_out=640),
    "one-adapter-back-again": dict(lengths=[9] * 40, adapter=[i % 2 for i in range(40)], n=2, R=17,
                                   n_in=160, n_out=96),
}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    S.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shape", FEW)
def test_few_tokens(shape, dt):
    c = ref.Case(dt, **FEW[shape])
    got = S.low_rank_add(c.yt, *c.args())
    ref.check(got, ref.add(c), "add")
    y = c.yt.clone(memory_format=torch.preserve_format)
    S.low_rank_add(y, *c.args(), out=y)
    assert torch.equal(y, got)
    idle = torch.ones(c.T, dtype=torch.bool, device="cuda")
    for t, _, _, _ in c.runs():
        idle[t] = False
    assert torch.equal(got[:, idle], c.yt[:, idle])
    ref.check(S.low_rank_project(c.W, *c.args()), ref.project(c), "project")


@pytest.mark.parametrize("dt", DTYPES)
def test_few_tokens_keep_their_infinities(dt):
    """One of two requests on the one adapter is not finite, the other clean."""
    c = ref.Case(dt, [3, 2, 4], [0, -1, 0], 1, 12, 200, 90, ranks=[7])
    clean = [S.low_rank_add(c.yt, *c.args()), S.low_rank_project(c.W, *c.args())]
    c.xt[5, :3] = float("nan")
    c.A[0, 7:] = float("inf")
    c.B[0, :, 7:] = float("nan")
    got = [S.low_rank_add(c.yt, *c.args()), S.low_rank_project(c.W, *c.args())]
    for g, w in zip(got, clean):
        assert torch.equal(g[:, 3:], w[:, 3:]) and g[:, :3].isnan().all()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shape", WIDE)
def test_project_row_tiles(shape, dt):
    c = ref.Case(dt, **WIDE[shape])
    ref.check(S.low_rank_project(c.W, *c.args()), ref.project(c))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shape", MANY)
def test_tiles(shape, dt):
    c = ref.Case(dt, **MANY[shape])
    ref.check(S.low_rank_add(c.yt, *c.args()), ref.add(c), "add")
    for name, g, w in zip(("dx", "dA", "dB"), S.low_rank_backward(c.dyt, *c.args()),
                          ref.backward(c)):
        ref.check(g, w, name)


def test_offsets_that_do_not_ascend_with_few_tokens():
    """Unspecified adapters, every access in bounds."""
    c = ref.Case("bf16", [5], [0], 1, 16, 128, 128)
    for off in ([-7, 9], [2 ** 31 - 1, -2 ** 31], [4, 1]):
        args = (c.xt, c.A, c.B, torch.tensor(off, dtype=torch.int32, device="cuda"), c.adapter,
                c.scale, c.ranks)
        assert S.low_rank_add(c.yt, *args).shape == c.yt.shape
        assert S.low_rank_project(c.W, *args).shape == c.yt.shape
    torch.cuda.synchronize()


def test_few_tokens_in_a_graph():
    c = ref.Case("bf16", [1], [1], 3, 16, 512, 320)
    S.low_rank_add(c.yt, *c.args())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = S.low_rank_add(c.yt, *c.args()), S.low_rank_project(c.W, *c.args())
    for ad in (2, 0, 1):
        c.adapter.fill_(ad)
        c.ad = [ad]
        graph.replay()
        torch.cuda.synchronize()
        ref.check(outs[0], ref.add(c), "add")
        ref.check(outs[1], ref.project(c), "project")


def test_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "low_rank_finetune.py")
    spec = importlib.util.spec_from_file_location("low_rank_finetune", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, norms, layer, dense = m.finetune()
    assert losses[-1] < 0.5 * losses[0] and all(n > 0 for n in norms)
    together, apart = m.serve(layer, dense)
    # fp32 sums of 512 + 8 terms in two orders, of a magnitude of |W| |x|
    assert (together - apart).abs().max() <= 2 * 2.0 ** -24 * 540 * 40
