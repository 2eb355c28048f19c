"""Refusals of the low-rank adapter and clipping calls, without a GPU: the C
entry points return a status before touching the device (pointers below are
never dereferenced), and the binding raises ValueError."""
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
    d = S.LowRankDesc(tokens=40, requests=3, adapters=2, rank=16, in_features=64, out_features=48,
                      dtype=2, A=FAKE, B=FAKE, offsets=FAKE, adapter=FAKE, ranks=None, scale=None)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def need(L, d, op):
    b = ctypes.c_size_t()
    assert L.spops_low_rank_workspace_size(ctypes.byref(d), op, ctypes.byref(b)) == 0
    return b.value


BAD_DESCS = [(dict(tokens=-1), 2), (dict(requests=-1), 2), (dict(adapters=0), 2),
             (dict(adapters=70000), 2), (dict(rank=0), 2), (dict(rank=257), 6),
             (dict(in_features=0), 2), (dict(out_features=0), 2),
             (dict(in_features=(1 << 24) + 1), 2), (dict(tokens=(1 << 30) + 1), 2),
             (dict(dtype=5), 3)]


@pytest.mark.parametrize("kw,code", BAD_DESCS)
def test_descriptor(L, kw, code):
    b, d = ctypes.c_size_t(), desc(**kw)
    big = 1 << 40
    assert L.spops_low_rank_workspace_size(ctypes.byref(d), 0, ctypes.byref(b)) == code
    for f in (L.spops_low_rank_add, L.spops_low_rank_project):
        assert f(ctypes.byref(d), FAKE, 64, FAKE, 64, FAKE, 64, FAKE, big, None) == code
    assert L.spops_low_rank_backward(ctypes.byref(d), FAKE, 64, FAKE, 64, FAKE, 64, FAKE, FAKE,
                                     FAKE, big, None) == code


def test_workspace_size(L):
    assert L.spops_low_rank_workspace_size(None, 0, ctypes.byref(ctypes.c_size_t())) == 1
    assert L.spops_low_rank_workspace_size(ctypes.byref(desc()), 0, None) == 1
    assert L.spops_low_rank_workspace_size(ctypes.byref(desc()), 3,
                                           ctypes.byref(ctypes.c_size_t())) == 6
    for op in range(3):
        assert need(L, desc(tokens=0), op) == 0
        # u alone: rank x tokens of f32
        assert need(L, desc(), op) >= 16 * 40 * 4


@pytest.mark.parametrize("op", [0, 1, 2])
def test_calls(L, op):
    name = ("add", "project", "backward")[op]
    f = getattr(L, "spops_low_rank_" + name)
    lead = 64 if op == 1 else 40
    grads = (FAKE, FAKE) if op == 2 else ()
    big = need(L, desc(), op)

    def call(d=None, first=FAKE, ldf=lead, x=FAKE, ldx=40, out=FAKE, ldo=40, g=grads, ws=FAKE,
             bytes_=big):
        return f(ctypes.byref(d or desc()), first, ldf, x, ldx, out, ldo, *g, ws, bytes_, None)

    assert f(None, FAKE, lead, FAKE, 40, FAKE, 40, *grads, FAKE, big, None) == 1
    assert call(ldf=lead - 1) == 2 and call(ldx=39) == 2 and call(ldo=39) == 2
    assert call(first=None) == 1 and call(x=None) == 1 and call(out=None) == 1
    for k in ("A", "B", "offsets", "adapter"):
        assert call(desc(**{k: None})) == 1
    assert call(ws=None) == 5 and call(bytes_=big - 1) == 5 and call(ws=FAKE + 16) == 5
    if op == 2:
        assert call(g=(None, FAKE)) == 1 and call(g=(FAKE, None)) == 1
    else:
        assert call(desc(tokens=0), first=None, x=None, out=None, ws=None, bytes_=0) == 0
    assert call(desc(tokens=1 << 30, in_features=1 << 24), ldf=1 << 30, ldx=1 << 30,
                ldo=1 << 30) == 2  # more tiles than one launch has


def test_clip_entry_point(L):
    b = ctypes.c_size_t()
    assert L.spops_clip_grad_norm_workspace_size(-1, ctypes.byref(b)) == 2
    assert L.spops_clip_grad_norm_workspace_size((1 << 20) + 1, ctypes.byref(b)) == 2
    assert L.spops_clip_grad_norm_workspace_size(3, None) == 1
    assert L.spops_clip_grad_norm_workspace_size(300, ctypes.byref(b)) == 0 and b.value > 0
    ok = dict(grad=FAKE, out=FAKE, numel=10, dtype=0)

    def call(count=2, max_norm=1.0, norm=FAKE, ws=FAKE, bytes_=b.value, null=False, **kw):
        ts = (S.ClipTensor * 2)(S.ClipTensor(**ok), S.ClipTensor(**{**ok, **kw}))
        return L.spops_clip_grad_norm(None if null else ts, count, max_norm, norm, ws, bytes_,
                                      None)

    assert call(count=-1) == 2 and call(count=1 << 21) == 2
    assert call(norm=None) == 1 and call(null=True) == 1
    assert call(max_norm=-1.0) == 9 and call(max_norm=float("nan")) == 9
    assert call(dtype=9) == 3 and call(numel=-1) == 2 and call(numel=(1 << 36) + 1) == 2
    assert call(grad=None) == 1 and call(out=None) == 1
    assert call(ws=None) == 5 and call(bytes_=8) == 5 and call(ws=FAKE + 4) == 5


def tensors(**kw):
    t = dict(first=torch.zeros(48, 40), xt=torch.zeros(64, 40), A=torch.zeros(2, 16, 64),
             B=torch.zeros(2, 48, 16), offsets=torch.zeros(4, dtype=torch.int32),
             adapter=torch.zeros(3, dtype=torch.int32), scale=torch.ones(2),
             ranks=torch.ones(2, dtype=torch.int32))
    t.update(kw)
    return list(t.values())


BAD_TENSORS = [
    (dict(xt=3), "xt must be a torch.Tensor"),
    (dict(xt=torch.zeros(64, 40, dtype=torch.float64)), "xt must be float32"),
    (dict(xt=torch.zeros(64)), "xt must be a matrix"),
    (dict(xt=torch.zeros(40, 64).t()), "unit stride"),
    (dict(xt=torch.zeros(1, 40).expand(64, 40)), "do not overlap"),
    (dict(xt=torch.zeros(64, 40).to_sparse()), "dense"),
    (dict(first=torch.zeros(48, 40, dtype=torch.float16)), "xt's dtype"),
    (dict(A=torch.zeros(2, 16, 64, dtype=torch.bfloat16)), "A must have xt's dtype"),
    (dict(B=torch.zeros(2, 48, 16, dtype=torch.bfloat16)), "B must have xt's dtype"),
    (dict(A=torch.zeros(16, 64)), "A must be adapters"),
    (dict(A=torch.zeros(2, 16, 65)), "A must be adapters"),
    (dict(A=torch.zeros(2, 64, 16).transpose(1, 2)), "A must be contiguous"),
    (dict(B=torch.zeros(3, 48, 16)), "B must be adapters"),
    (dict(B=torch.zeros(2, 48, 15)), "B must be adapters"),
    (dict(offsets=torch.zeros(4, dtype=torch.int64)), "offsets must be a vector of int32"),
    (dict(offsets=torch.zeros(3, dtype=torch.int32)), "one entry more"),
    (dict(adapter=torch.zeros(3, 1, dtype=torch.int32)), "adapter must be a vector"),
    (dict(adapter=torch.zeros(6, dtype=torch.int32)[::2]), "adapter must be contiguous"),
    (dict(scale=torch.ones(3)), "scale must be"),
    (dict(scale=torch.ones(2, dtype=torch.float64)), "scale must be"),
    (dict(ranks=torch.ones(2)), "ranks must be"),
    (dict(), "must be a GPU tensor"),
]


@pytest.mark.parametrize("kw,message", BAD_TENSORS)
def test_binding(L, kw, message):
    for f in (P.low_rank_add, P.low_rank_backward):
        with pytest.raises(ValueError, match=message):
            f(*tensors(**kw))
    kw.setdefault("first", torch.zeros(48, 64))
    if kw["first"].shape == (48, 64):
        with pytest.raises(ValueError, match=message):
            P.low_rank_project(*tensors(**kw))


def test_binding_shapes_of_the_first_matrix_and_out(L):
    for f in (P.low_rank_add, P.low_rank_backward):
        with pytest.raises(ValueError, match="out_features x tokens"):
            f(*tensors(first=torch.zeros(48, 41)))
    with pytest.raises(ValueError, match="out_features x in_features"):
        P.low_rank_project(*tensors(first=torch.zeros(48, 63)))
    with pytest.raises(ValueError, match="out must be out_features x tokens"):
        P.low_rank_add(*tensors(), out=torch.zeros(48, 39))
    with pytest.raises(ValueError, match="out must have xt's dtype"):
        P.low_rank_add(*tensors(), out=torch.zeros(48, 40, dtype=torch.float16))


def test_clip_binding(L):
    g = [torch.zeros(4), torch.zeros(3, dtype=torch.bfloat16)]
    for grads, out, message in [
            ([], None, "at least one tensor"),
            ([1], None, "must be a torch.Tensor"),
            ([torch.zeros(4, dtype=torch.float64)], None, "must be float32"),
            ([torch.zeros(4, 4).t()], None, "must be contiguous"),
            (g, g[:1], "one tensor per gradient"),
            (g, [g[0], torch.zeros(3)], "dtype and size"),
            (g, [g[0], torch.zeros(2, dtype=torch.bfloat16)], "dtype and size"),
            (g, None, "must be a GPU tensor")]:
        with pytest.raises(ValueError, match=message):
            P.clip_grad_norm(grads, 1.0, out=out)
    with pytest.raises(TypeError):
        P.clip_grad_norm(g, "1")
    with pytest.raises(TypeError):
        P.clip_grad_norm(None, 1.0)
