"""Calls of more workgroups than one launch has work-items for (2^32)."""
import pytest
import torch

import unstructured_sparse_linear_amd as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    S.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def integers(g, most, *shape):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(torch.bfloat16)


def test_gradients_of_the_largest_pool():
    """65535 adapters: 2 x 129 blocks of features times the pool, of 256 threads."""
    n, n_in, n_out, T = 65535, 8256, 8256, 9
    g = torch.Generator(device="cuda").manual_seed(0)
    A = torch.ones(n, 1, n_in, dtype=torch.bfloat16, device="cuda")
    B = torch.ones(n, n_out, 1, dtype=torch.bfloat16, device="cuda")
    xt, dyt = integers(g, 1, n_in, T), integers(g, 1, n_out, T)
    off = torch.tensor([0, 2, 5, 5, 9], dtype=torch.int32, device="cuda")
    which = [65534, 0, 7, 40_000]
    dx, dA, dB = S.low_rank_backward(dyt, xt, A, B, off,
                                     torch.tensor(which, dtype=torch.int32, device="cuda"))
    u, du = xt.double().sum(0), dyt.double().sum(0)  # exact integers below 8256
    assert torch.equal(dx.double(), du.to(torch.bfloat16).double().expand(n_in, T))
    used = 0
    for a, t in ((65534, slice(0, 2)), (0, slice(2, 5)), (40_000, slice(5, 9))):
        wA = (xt[:, t].double() * du[t]).sum(1).to(torch.bfloat16)
        wB = (dyt[:, t].double() * u[t]).sum(1).to(torch.bfloat16)
        assert torch.equal(dA[a, 0], wA) and torch.equal(dB[a, :, 0], wB)
        used += int(wA.count_nonzero()) + int(wB.count_nonzero())
    assert int(dA.count_nonzero()) + int(dB.count_nonzero()) == used


def test_project_of_many_tokens():
    """Blocks of 48 rows times tiles of 64 tokens, of 768 threads."""
    n_in, n_out, T = 8, 131_072, 137_000
    assert (n_out // 48) * (T // 64) * 768 > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    W, xt = integers(g, 3, n_out, n_in), integers(g, 3, n_in, T)
    A, B = integers(g, 2, 2, 1, n_in), integers(g, 2, 2, n_out, 1)
    off = torch.tensor([0, 70_001, T], dtype=torch.int32, device="cuda")
    ad = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    y = S.low_rank_project(W, xt, A, B, off, ad)
    u = torch.cat([A[1].float() @ xt[:, :70_001].float(), A[0].float() @ xt[:, 70_001:].float()], 1)
    second = torch.arange(T, device="cuda") >= 70_001
    for r in range(0, n_out, 4096):
        rows = slice(r, r + 4096)
        want = W[rows].float() @ xt.float()  # integers below 72 + 2 x 48: exact in bf16
        want += torch.where(second, B[0, rows].float() * u, B[1, rows].float() * u)
        assert torch.equal(y[rows], want.to(torch.bfloat16))
