"""Low-rank adapters over many tokens, exactly: inputs are small integers whose
sums stay below 2^24, so every output is the float64 result rounded once.  The
gradients list an adapter's tokens 8192 at a time; adapters here have theirs in
the first list, across two, and in later ones alone."""
import pytest
import torch

import unstructured_sparse_linear_amd as S
import lowrank_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    S.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def lengths_of(T):
    """Requests of adapters 0 (early), 1 (across 8192), none, 2 (the tail alone), 0."""
    cut = [0, 5000, min(T - 4, 8250), min(T - 3, 8300), T - 2, T]
    return [b - a for a, b in zip(cut, cut[1:])], [0, 1, -1, 2, 0]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R", [5, 20, 40])
@pytest.mark.parametrize("T", [8191, 8192, 8193, 8225, 16_384, 16_385, 24_600])
def test_token_lists(T, R, dt):
    lengths, adapter = lengths_of(T)
    c = ref.Case(dt, lengths, adapter, 4, R, 40, 24, ranks=[R, R - 1, 3, R])
    g = torch.Generator().manual_seed(T + R)
    for name in ("A", "B", "xt", "yt", "dyt", "W"):
        t = getattr(c, name)
        t.copy_(torch.randint(-1, 2, t.shape, generator=g))
    c.scale = torch.tensor([1.0, 2.0, 0.5, 1.0], device="cuda")
    add, project = c.yt.double(), ref.mm(c.W.double(), c.xt.double())
    dx = torch.zeros_like(c.xt, dtype=torch.float64)
    dA, dB = torch.zeros_like(c.A, dtype=torch.float64), torch.zeros_like(c.B, dtype=torch.float64)
    for t, a, k, s in c.runs():
        x, dy = c.xt[:, t].double(), c.dyt[:, t].double()
        A, B = c.A[a, :k].double(), c.B[a, :, :k].double()
        u, du = s * ref.mm(A, x), s * ref.mm(B.t(), dy)
        add[:, t] += ref.mm(B, u)
        project[:, t] += ref.mm(B, u)
        dx[:, t] = ref.mm(A.t(), du)
        dA[a, :k] += ref.mm(du, x.t())
        dB[a, :, :k] += ref.mm(dy, u.t())
    for want in (add, project, dx, dA, dB):
        assert want.abs().max() < 60_000
    # every adapter's gradient is there and differs from its first list's alone
    for a in range(3):
        assert dA[a].any() and dB[a].any()
    got = (S.low_rank_add(c.yt, *c.args()), S.low_rank_project(c.W, *c.args()),
           *S.low_rank_backward(c.dyt, *c.args()))
    for name, v, want in zip(("add", "project", "dx", "dA", "dB"), got,
                             (add, project, dx, dA, dB)):
        assert torch.equal(v, want.to(v.dtype)), name


def test_gradients_past_32_bits():
    """x, dy and dx of more than 2^31 values, rows of odd length: all of dA and dB,
    and dx on tokens from both ends."""
    T, n_in, n_out, R = 262_147, 8200, 8200, 4
    g = torch.Generator(device="cuda").manual_seed(2)

    def ternary(*shape):
        t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        for rows in t.split(512):
            rows.copy_(torch.randint(-1, 2, rows.shape, generator=g, device="cuda",
                                     dtype=torch.int8))
        return t

    xt, dyt = ternary(n_in, T), ternary(n_out, T)
    assert xt.numel() > 2 ** 31
    A, B = ternary(2, R, n_in), ternary(2, n_out, R)
    cut = 200_003
    off = torch.tensor([0, cut, T], dtype=torch.int32, device="cuda")
    ad = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    dx, dA, dB = S.low_rank_backward(dyt, xt, A, B, off, ad)
    wA = torch.zeros(2, R, n_in, dtype=torch.float64, device="cuda")
    wB = torch.zeros(2, n_out, R, dtype=torch.float64, device="cuda")
    for a, lo, hi in ((1, 0, cut), (0, cut, T)):
        for t in range(lo, hi, 32_768):
            x, dy = xt[:, t:min(t + 32_768, hi)].double(), dyt[:, t:min(t + 32_768, hi)].double()
            u, du = ref.mm(A[a].double(), x), ref.mm(B[a].double().t(), dy)
            assert max(u.abs().max(), du.abs().max()) < 2 ** 16
            wA[a] += ref.mm(du, x.t())
            wB[a] += ref.mm(dy, u.t())
    assert max(wA.abs().max(), wB.abs().max()) < 2 ** 22
    assert wA.abs().mean() > 1000 and wB.abs().mean() > 1000
    assert torch.equal(dA, wA.to(dA.dtype)) and torch.equal(dB, wB.to(dB.dtype))
    for a, at in ((1, [0, 1, 77_777, cut - 1]), (0, [cut, T - 2, T - 1])):
        du = ref.mm(B[a].double().t(), dyt[:, at].double())
        want = ref.mm(A[a].double().t(), du)
        assert torch.equal(dx[:, at], want.to(dx.dtype))
