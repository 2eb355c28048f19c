"""Refusals of the 4-bit matrix and dropout calls, without a GPU: the C entry points
return a status before touching the device (pointers below are never dereferenced),
and the binding raises ValueError."""
import ctypes
import os

import pytest
import torch

import unstructured_sparse_linear_amd as P
from unstructured_sparse_linear_amd import spops as S

FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    if not (os.path.exists(S.LIB_PATH)
            and os.path.exists(os.path.join(os.path.dirname(S.LIB_PATH), "_marshal.so"))):
        from unstructured_sparse_linear_amd import build
        build.build()
    return S.lib()


def desc(**kw):
    d = S.Mx4Desc(rows=300, cols=200, codes=FAKE, scales=FAKE)
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


def test_quantize_entry_point(L):
    f = L.spops_mx4_quantize
    ok = [FAKE, 0, 30, 40, 40, 1, FAKE, FAKE, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call(_1=7) == 3
    assert call(_2=0) == 2 and call(_3=0) == 2 and call(_2=-1) == 2
    assert call(_2=(1 << 24) + 1) == 2 and call(_3=(1 << 24) + 1, _4=1 << 25) == 2
    assert call(_4=39) == 2                        # rows that overlap
    assert call(_5=2) == 2                         # neither stride is one
    assert call(_4=1, _5=29) == 2                  # columns that overlap
    assert call(_0=None) == 1 and call(_6=None) == 1 and call(_7=None) == 1
    assert call(_6=FAKE + 8) == 2                  # codes not aligned


BAD = [(dict(rows=0), 2), (dict(cols=0), 2), (dict(rows=(1 << 24) + 1), 2),
       (dict(cols=(1 << 24) + 1), 2), (dict(codes=None), 1), (dict(scales=None), 1),
       (dict(codes=FAKE + 4), 2)]


@pytest.mark.parametrize("kw,code", BAD)
def test_descriptor(L, kw, code):
    big = 1 << 40
    assert L.spops_mx4_dequantize(desc(**kw), FAKE, 0, 1 << 25, None) == code
    assert L.spops_mx4_matmul(desc(**kw), 0, FAKE, 0, 5, 5, FAKE, 5, FAKE, big, None) == code
    assert L.spops_mx4_matmul4(desc(**kw), desc(), FAKE, 0, 1 << 25, FAKE, big, None) == code
    assert L.spops_mx4_matmul4(desc(), desc(**kw), FAKE, 0, 1 << 25, FAKE, big, None) == code


def test_dequantize_entry_point(L):
    f = L.spops_mx4_dequantize
    assert f(None, FAKE, 0, 200, None) == 1
    assert f(desc(), FAKE, 5, 200, None) == 3
    assert f(desc(), FAKE, 0, 199, None) == 2
    assert f(desc(), None, 0, 200, None) == 1


def test_matmul_entry_point(L):
    b = ctypes.c_size_t()
    size = L.spops_mx4_matmul_workspace_size
    assert size(None, 0, 0, 5, ctypes.byref(b)) == 1 and size(desc(), 0, 0, 5, None) == 1
    assert size(desc(), 0, 9, 5, ctypes.byref(b)) == 3
    assert size(desc(), 0, 0, -1, ctypes.byref(b)) == 2
    assert size(desc(), 0, 0, (1 << 30) + 1, ctypes.byref(b)) == 2
    assert size(desc(rows=1 << 24), 0, 0, 1 << 30, ctypes.byref(b)) == 2
    assert size(desc(), 0, 0, 0, ctypes.byref(b)) == 0 and b.value == 0
    f = L.spops_mx4_matmul
    for transposed in (0, 1):
        assert size(desc(cols=4096, rows=4096), transposed, 2, 40, ctypes.byref(b)) == 0
        need, d = b.value, desc(cols=4096, rows=4096)
        ok = [d, transposed, FAKE, 2, 40, 40, FAKE, 40, FAKE, need, None]

        def call(**kw):
            a = list(ok)
            for k, v in kw.items():
                a[int(k[1:])] = v
            return f(*a)

        assert call(_0=None) == 1 and call(_3=4) == 3
        assert call(_4=-1) == 2 and call(_5=39) == 2 and call(_7=39) == 2
        assert call(_2=None) == 1 and call(_6=None) == 1
        assert call(_4=0, _2=None, _6=None) == 0      # no tokens: nothing to do
        if need:
            assert call(_8=None) == 5 and call(_9=need - 1) == 5 and call(_8=FAKE + 16) == 5


def test_matmul4_entry_point(L):
    b = ctypes.c_size_t()
    size = L.spops_mx4_matmul4_workspace_size
    assert size(None, 5, ctypes.byref(b)) == 1 and size(desc(), 5, None) == 1
    assert size(desc(), -1, ctypes.byref(b)) == 2
    assert size(desc(), (1 << 24) + 1, ctypes.byref(b)) == 2
    wide = dict(cols=4096)
    assert size(desc(**wide), 40, ctypes.byref(b)) == 0
    f, need, x = L.spops_mx4_matmul4, b.value, desc(rows=40, **wide)
    assert f(desc(**wide), x, FAKE, 7, 40, FAKE, need, None) == 3
    assert f(None, x, FAKE, 0, 40, FAKE, need, None) == 1
    assert f(desc(**wide), None, FAKE, 0, 40, FAKE, need, None) == 1
    assert f(desc(), x, FAKE, 0, 40, FAKE, need, None) == 2         # inner sizes differ
    assert f(desc(**wide), x, FAKE, 0, 39, FAKE, need, None) == 2
    assert f(desc(**wide), x, None, 0, 40, FAKE, need, None) == 1
    if need:
        assert f(desc(**wide), x, FAKE, 0, 40, FAKE, need - 1, None) == 5
        assert f(desc(**wide), x, FAKE, 0, 40, None, need, None) == 5


def test_dropout_entry_point(L):
    f = L.spops_dropout
    ok = [FAKE, 0, 30, 40, 40, FAKE, 40, 0.5, 1, 2, None, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call(_1=3) == 3
    assert call(_2=-1) == 2 and call(_3=-1) == 2 and call(_4=39) == 2 and call(_6=39) == 2
    assert call(_2=1 << 31) == 2 and call(_3=1 << 31, _4=1 << 31, _6=1 << 31) == 2
    for p in (-0.01, 1.01, float("nan")):
        assert call(_7=p) == 9
    assert call(_0=None) == 1 and call(_5=None) == 1
    assert call(_2=0, _0=None, _5=None) == 0 and call(_3=0, _0=None, _5=None) == 0


def mx4(rows=6, cols=70):
    nb = (cols + 31) // 32
    return P.Mx4Matrix(torch.zeros(rows, 16 * nb, dtype=torch.uint8),
                       torch.zeros(rows, nb, dtype=torch.uint8), cols)


def test_matrix():
    W = mx4()
    assert W.shape == (6, 70) and "6 x 70" in repr(W)
    for codes, scales, cols in [
            (W.codes.int(), W.scales, 70), (W.codes, W.scales.int(), 70),
            (W.codes, W.scales, 64), (W.codes, W.scales, 97), (W.codes, W.scales, 0),
            (W.codes[0], W.scales, 70), (W.codes, W.scales[:5], 70), (W.codes[:0], W.scales[:0], 70),
            (torch.zeros(48, 6, dtype=torch.uint8).t(), W.scales, 70)]:
        with pytest.raises(ValueError):
            P.Mx4Matrix(codes, scales, cols)


@pytest.mark.parametrize("w,message", [
    (3, "must be a torch.Tensor"),
    (torch.zeros(4, 4, dtype=torch.float64), "must be float32"),
    (torch.zeros(4), "must be a matrix"),
    (torch.zeros(0, 4), "must not be empty"),
    (torch.zeros(4, 8)[:, ::2], "unit stride"),
    (torch.zeros(1, 4).expand(3, 4), "unit stride"),
    (torch.zeros(4, 4).to_sparse(), "dense"),
    (torch.zeros(4, 4), "must be a GPU tensor")])
def test_quantize_binding(L, w, message):
    with pytest.raises(ValueError, match=message):
        P.mx4_quantize(w)


def test_products_binding(L):
    W, x = mx4(), torch.zeros(70, 5)
    for args, kw, message in [
            ((W, torch.zeros(71, 5)), {}, "columns x tokens"),
            ((W, torch.zeros(70, 5)), dict(transposed=True), "rows x tokens"),
            ((W, torch.zeros(70)), {}, "must be a matrix"),
            ((W, torch.zeros(5, 70).t()), {}, "unit stride"),
            ((W, torch.zeros(70, 5, dtype=torch.float64)), {}, "must be float32"),
            ((W, 5), {}, "must be a torch.Tensor"),
            ((W, x), dict(out_dtype=torch.float16), "dtype of xt"),
            ((W, x), {}, "must be a GPU tensor"),
            ((W, mx4(5, 70)), dict(transposed=True), "transposed"),
            ((W, mx4(5, 71)), {}, "W's columns"),
            ((W, mx4(5, 70)), dict(out_dtype=torch.float64), "dtype must be"),
            ((W, mx4(5, 70)), {}, "must be a GPU tensor")]:
        with pytest.raises(ValueError, match=message):
            P.mx4_matmul(*args, **kw)
    with pytest.raises(ValueError, match="dtype must be"):
        P.mx4_dequantize(W, torch.float64)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        P.mx4_dequantize(W)


def test_dropout_binding(L):
    x = torch.zeros(4, 6)
    for args, kw, message in [
            ((5, 0.1, 1), {}, "Tensor|requires_grad"),
            ((x.double(), 0.1, 1), {}, "must be float32"),
            ((x.t(), 0.1, 1), {}, "unit stride"),
            ((torch.zeros(2, 3, 4).transpose(0, 1), 0.1, 1), {}, "contiguous or a matrix"),
            ((x, -0.1, 1), {}, "between 0 and 1"),
            ((x, float("nan"), 1), {}, "between 0 and 1"),
            ((x, 0.1, torch.zeros(2)), {}, "int64 vector"),
            ((x, 0.1, torch.zeros(3, dtype=torch.int64)), {}, "int64 vector"),
            ((x, 0.1, torch.zeros(4, dtype=torch.int64)[::2]), {}, "must be contiguous"),
            ((x, 0.1, 1), dict(out=torch.zeros(4, 5)), "dtype and shape"),
            ((x, 0.1, 1), dict(out=torch.zeros(4, 6).half()), "dtype and shape"),
            ((torch.zeros(4, 6, requires_grad=True), 0.1, 1), dict(out=torch.zeros(4, 6)),
             "no gradient"),
            ((torch.zeros(4, 6), 0.1, 1), {}, "must be a GPU tensor")]:
        with pytest.raises((ValueError, AttributeError), match=message):
            P.dropout(*args, **kw)
    with pytest.raises(TypeError):
        P.dropout(torch.zeros(4, 6), "p", 1)
    with pytest.raises(TypeError):
        P.dropout(torch.zeros(4, 6), 0.1, 1.5)
    with pytest.raises(ValueError, match="dropout must be"):
        P.LowRankAdapters(1, 2, 4, 4, device="cpu", dropout=1.5)


def test_adapters_keep_their_state():
    """Without dropout nothing is added to the module; with it a seed and a step."""
    plain = P.LowRankAdapters(1, 2, 4, 4, device="cpu")
    assert sorted(plain.state_dict()) == ["A", "B"]
    drop = P.LowRankAdapters(1, 2, 4, 4, device="cpu", dropout=0.1, seed=5)
    assert drop.dropout_state.tolist() == [5, 0]
    assert drop.half().dropout_state.dtype == torch.int64 and drop.A.dtype == torch.float16
    torch.manual_seed(0)
    a = P.LowRankAdapters(1, 2, 4, 4, device="cpu", dropout=0.1)
    assert a.dropout_state[0] != P.LowRankAdapters(1, 2, 4, 4, device="cpu",
                                                   dropout=0.1).dropout_state[0]
