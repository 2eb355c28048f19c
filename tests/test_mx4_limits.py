"""The largest outputs of the 4-bit products: 2^23 tiles of 128 x 128, and fewer of f32,
whose tiles have 512 threads (a launch has fewer than 2^32)."""
import ctypes

import pytest
import torch

import mx4_ref as ref
import unstructured_sparse_linear_amd as P
from test_mx4_refusals import FAKE, L, desc  # noqa: F401

MOST = 1 << 30  # tokens


@pytest.mark.parametrize("transposed", [0, 1])
def test_limit(L, transposed):  # noqa: F811
    bytes_, size = ctypes.c_size_t(), L.spops_mx4_matmul_workspace_size

    def status(features, tokens, dtype):
        one = dict(cols=features, rows=5) if transposed else dict(rows=features, cols=5)
        return size(desc(**one), transposed, dtype, tokens, ctypes.byref(bytes_))

    for dtype in range(3):
        f32 = dtype == 0
        # a row of tiles, and rows and columns of them
        assert status(128, MOST, dtype) == (2 if f32 else 0)
        assert status(128, MOST - 128, dtype) == 0
        assert status(129, MOST // 2, dtype) == (2 if f32 else 0)
        assert status(129, MOST // 2 - 128, dtype) == 0
        assert status(129, MOST // 2 + 1, dtype) == 2
        assert status(1 << 24, 8192, dtype) == (2 if f32 else 0)
        assert status(1 << 24, 8064, dtype) == 0
        assert status(1 << 24, 8193, dtype) == 2
        f = L.spops_mx4_matmul
        d = desc(cols=129, rows=5) if transposed else desc(rows=129, cols=5)
        t = MOST // 2 + (0 if f32 else 1)
        assert f(d, transposed, FAKE, dtype, t, t, FAKE, t, None, 0, None) == 2


def test_limit_of_two(L):  # noqa: F811
    """The product of two 4-bit matrices has 256 threads a tile in every type."""
    size, b = L.spops_mx4_matmul4_workspace_size, ctypes.c_size_t()
    assert size(desc(rows=1 << 24), 8192, ctypes.byref(b)) == 0
    assert size(desc(rows=1 << 24), 8193, ctypes.byref(b)) == 2
    x = desc(rows=8193)
    assert L.spops_mx4_matmul4(desc(rows=1 << 24), x, FAKE, 0, 8193, FAKE, 1 << 40, None) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,tokens", [("f32", MOST - 128), ("bf16", MOST)])
@pytest.mark.parametrize("transposed", [False, True])
def test_largest_output(dtype, tokens, transposed):
    """As many tiles as are accepted, of one feature: each value doubled."""
    W = P.mx4_quantize(torch.full((1, 1), 2.0, device="cuda"))
    x = torch.arange(tokens, dtype=torch.int32, device="cuda").remainder_(251)
    x = x.to(ref.DTYPES[dtype]).reshape(1, -1)
    y = P.mx4_matmul(W, x, transposed=transposed)
    assert torch.equal(y, x.mul_(2))
    del x, y
    torch.cuda.empty_cache()
