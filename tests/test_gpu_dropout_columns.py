"""Dropout between columns of one larger matrix: what does not overlap is taken, what
does is refused."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import unstructured_sparse_linear_amd as S
from test_gpu_dropout import _gpu, expected, values  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("left,right", [(0, 37), (37, 0), (1, 38), (40, 3), (63, 0), (3, 63)])
def test_columns_side_by_side(dtype, left, right):
    """x and out beside each other, at odd addresses too; what lies around them stays."""
    wide = 37
    big, v = values((50, 101), dtype)
    x, out = big[:, left:left + wide], big[:, right:right + wide]
    want = big.clone()
    want[:, right:right + wide] = expected(v[:, left:left + wide], 0.3, 9, 2, dtype).cuda()
    assert S.dropout(x, 0.3, 9, 2, out=out) is out
    assert torch.equal(big, want)


def test_columns_that_end_in_the_next_row():
    """Windows whose rows reach past the end of the larger matrix's."""
    flat, v = values((40 * 50 + 60,), "f32")
    x = flat.as_strided((40, 25), (50, 1), 30)
    out = flat.as_strided((40, 25), (50, 1), 55)
    keep = v[30:30 + 40 * 50].reshape(40, 50)[:, :25]
    S.dropout(x, 0.3, 9, 2, out=out)
    assert torch.equal(out.cpu(), expected(keep, 0.3, 9, 2, "f32"))
    assert torch.equal(x.cpu().double(), torch.from_numpy(keep))


def test_overlaps_are_refused():
    flat, _ = values((3000,), "f32")
    before = flat.clone()

    def matrix(at, rows, cols, lead):
        return flat.as_strided((rows, cols), (lead, 1), at)

    for x, out in [(matrix(0, 20, 30, 50), matrix(29, 20, 30, 50)),     # one column
                   (matrix(29, 20, 30, 50), matrix(0, 20, 30, 50)),
                   (matrix(0, 20, 30, 50), matrix(35, 20, 30, 50)),     # round the row's end
                   (matrix(0, 20, 30, 50), matrix(50, 20, 30, 50)),     # a row further
                   (matrix(0, 20, 30, 50), matrix(0, 20, 30, 60)),      # other distances
                   (matrix(0, 20, 30, 30), matrix(570, 20, 30, 30)),    # the last row
                   (matrix(0, 1, 30, 50), matrix(10, 1, 30, 50)),
                   (flat[:1000], flat[500:1500]),
                   (flat[:1000].view(10, 10, 10), flat[1:1001].view(10, 10, 10))]:
        with pytest.raises(ValueError, match="out must be x or not overlap it"):
            S.dropout(x, 0.5, 1, out=out)
    assert torch.equal(flat, before)
    # one row each, side by side
    x, out = matrix(0, 1, 30, 50), matrix(30, 1, 30, 50)
    S.dropout(x, 0.5, 1, out=out)
    assert np.array_equal(out.cpu().double().numpy(),
                          ref.dropout(x.cpu().double().numpy(), 0.5, 1, 0))
