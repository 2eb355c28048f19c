"""4-bit products and values at the edges of what f16 holds: scales of 104 and 140, every
scale dequantised to f16, and large tiles of which only some hold scales past them."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import unstructured_sparse_linear_amd as S
from test_gpu_mx4 import f64
from test_gpu_mx4_paths import _gpu, whole_matrix, whole_numbers  # noqa: F401

pytestmark = pytest.mark.gpu


def test_every_element_and_scale_in_f16():
    """What f16 holds exactly, subnormals included; the nearest of the others, or an
    infinity."""
    i = np.tile(np.arange(16, dtype=np.uint8), 2)
    codes = np.repeat((i[0::2] | (i[1::2] << 4))[None], 256, 0)
    scales = np.arange(256, dtype=np.uint8)[:, None]
    W = S.Mx4Matrix(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 32)
    values = ref.dequantize(codes, scales, 32)
    with np.errstate(over="ignore"):
        half = values.astype(np.float16).astype(np.float64)
    assert np.array_equal(half[104:141], values[104:141])
    assert np.array_equal(f64(S.mx4_dequantize(W, torch.float16)), half, equal_nan=True)


# few tokens, small and large tiles
SIZES = [(96, 160, 1), (96, 160, 20), (4100, 96, 60), (200, 520, 150), (2100, 300, 2100),
         (4097, 300, 2011)]


@pytest.mark.parametrize("low,high,power", [(104, 104, 14), (104, 107, 14), (137, 140, -12),
                                            (140, 140, -13)])
@pytest.mark.parametrize("rows,cols,tokens", SIZES)
@pytest.mark.parametrize("transposed", [False, True])
def test_edges_of_f16(low, high, power, rows, cols, tokens, transposed):
    """W in f16 is subnormal (from 2^-24 on) or up to 49152; x is a whole number of -3..3
    times a power of two.  Sums are at most 2^24 times the smallest product, so f32 holds
    them exactly and each output is rounded once."""
    W, w = whole_matrix([low, rows], rows, cols, low, high)
    m = w.t().contiguous() if transposed else w
    x = whole_numbers((m.shape[1], tokens), "f16", low) * 2.0 ** power
    assert x.dtype == torch.float16
    smallest = 2.0 ** (low - 128 + power)
    assert float(torch.mm(m.abs(), x.double().abs()).max()) < 2 ** 24 * smallest
    want = torch.mm(m, x.double()).half()
    assert torch.equal(S.mx4_matmul(W, x, transposed=transposed), want)


@pytest.mark.parametrize("tokens", [2011, 2176, 1990])
def test_wide_blocks_in_some_large_tiles(tokens):
    """Tiles of 256 x 128, whole and in pieces: those with a scale that f16 does not hold
    take x in two parts, one buffer of it, the others run on f16."""
    rows, cols = 4097, 530
    W, _ = whole_matrix(6, rows, cols, low=118, high=121)
    # rows of tiles 0, 3 and 16 (the one row past the last whole tile), the last block of
    # a row and the first
    W.scales[5, 16] = W.scales[3 * 256 + 255, 0] = W.scales[4096, 7] = 90
    w = S.mx4_dequantize(W).double()
    x = whole_numbers((cols, tokens), "f16", 6)
    want, size = torch.mm(w, x.double()), torch.mm(w.abs(), x.double().abs())
    limit = torch.from_numpy(ref.bound(want.cpu().numpy(), cols, size.cpu().numpy(), "f16")).cuda()
    got = [S.mx4_matmul(W, x) for _ in range(3)]
    assert ((got[0].double() - want).abs() <= limit).all()
    assert torch.equal(got[1], got[0]) and torch.equal(got[2], got[0])
    # and where every tile is one of them
    W.scales[::128, ::4] = 90
    w = S.mx4_dequantize(W).double()
    want, size = torch.mm(w, x.double()), torch.mm(w.abs(), x.double().abs())
    limit = torch.from_numpy(ref.bound(want.cpu().numpy(), cols, size.cpu().numpy(), "f16")).cuda()
    assert ((S.mx4_matmul(W, x).double() - want).abs() <= limit).all()
