"""Gradient norm and clipping on the GPU against float64."""
import math

import pytest
import torch

import unstructured_sparse_linear_amd as S
from lowrank_ref import DT, TINY

pytestmark = pytest.mark.gpu

SIZES = {
    "one-element": [1],
    "one": [1000],
    "odd": [1, 7, 8191, 8192, 8193, 3, 100_001],
    "empty-among": [0, 5, 0, 0, 4097, 0],
    "table-full": [33 + i for i in range(128)],
    "table-over": [1 + 5 * i for i in range(129)],
    "many": [1 + (977 * i) % 3001 for i in range(300)],
    "large": [30_000_001, 12],
}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    S.lib()
    yield
    torch.cuda.synchronize()


def make(sizes, dt, std=1.0, seed=0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kinds = ["f32", "bf16", "f16"] if dt == "mixed" else [dt]
    out = []
    for i, s in enumerate(sizes):
        t = torch.randn(s + shift, generator=g, device="cuda") * std
        out.append(t.to(DT[kinds[i % len(kinds)]])[shift:])
    return out


def check(grads, outs, norm, max_norm):
    """norm: fp64 sums, one fp32 rounding.  out: the factor in fp32, the fp32
    product and the rounding to the storage type, half a step each."""
    want = math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))
    assert abs(float(norm) - want) <= 2.0 ** -24 * want * (1 + 1e-6)
    coef = min(1.0, max_norm / (want + 1e-6))
    for g, o in zip(grads, outs):
        eps = torch.finfo(g.dtype).eps / 2
        tiny = TINY[{v: k for k, v in DT.items()}[g.dtype]]
        ref = g.double() * coef
        bound = (eps + 2.01 * 2.0 ** -24) * ref.abs() + 2 * tiny
        assert ((o.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES)
def test_clip(sizes, dt):
    grads = make(SIZES[sizes], dt)
    kept = [g.clone() for g in grads]
    for max_norm in (0.5, 1e9, 0.0):
        outs = [torch.full_like(g, 7.0) for g in grads]
        norm = S.clip_grad_norm(grads, max_norm, out=outs)
        assert norm.shape == () and norm.dtype == torch.float32
        check(grads, outs, norm, max_norm)
        for g, k in zip(grads, kept):
            assert torch.equal(g, k)
        if max_norm == 1e9:
            for g, o in zip(grads, outs):
                assert torch.equal(g, o)
        again = [torch.empty_like(g) for g in grads]
        assert torch.equal(norm, S.clip_grad_norm(tuple(grads), max_norm, out=again))
        for a, o in zip(again, outs):
            assert torch.equal(a, o)
        inplace = [g.clone() for g in grads]
        S.clip_grad_norm(inplace, max_norm)
        for a, o in zip(inplace, outs):
            assert torch.equal(a, o)


def test_unaligned_slices():
    """Gradients and outputs that start off the 16-byte grid; neighbours kept."""
    grads = make([4096, 8195, 20_000], "bf16", shift=3)
    flat = torch.full((sum(g.numel() for g in grads) + 2,), 7.0, dtype=torch.bfloat16,
                      device="cuda")
    outs, at = [], 1
    for g in grads:
        outs.append(flat[at:at + g.numel()])
        at += g.numel()
    norm = S.clip_grad_norm(grads, 1.0, out=outs)
    check(grads, outs, norm, 1.0)
    assert flat[0] == 7.0 and flat[-1] == 7.0


@pytest.mark.parametrize("std", [1e-30, 1e25])
def test_squares_outside_fp32(std):
    grads = make([5000, 17], "f32", std=std)
    outs = [torch.empty_like(g) for g in grads]
    norm = S.clip_grad_norm(grads, 1.0, out=outs)
    check(grads, outs, norm, 1.0)


def test_not_finite():
    """An infinite norm scales by zero (infinity itself gives NaN); NaN spreads."""
    grads = make([100, 9000], "f32")
    grads[1][77] = float("inf")
    outs = [torch.empty_like(g) for g in grads]
    assert S.clip_grad_norm(grads, 1.0, out=outs) == float("inf")
    assert not outs[0].any() and outs[1][77].isnan() and not outs[1][:77].any()
    grads[0][3] = float("nan")
    assert S.clip_grad_norm(grads, 1e9, out=outs).isnan()
    assert all(o.isnan().all() for o in outs)
    S.clip_grad_norm(grads, 1e9)
    assert all(g.isnan().all() for g in grads)
    zeros = [torch.zeros(10, device="cuda")]
    assert S.clip_grad_norm(zeros, 0.0) == 0 and not zeros[0].any()
    grads = make([64], "f32")
    assert torch.isfinite(S.clip_grad_norm(grads, float("inf")))


def test_past_32_bits():
    g = torch.full((2 ** 31 + 70_001,), 0.5, dtype=torch.bfloat16, device="cuda")
    g[-1] = 2.0
    want = math.sqrt(0.25 * (g.numel() - 1) + 4.0)
    norm = S.clip_grad_norm([g], want / 4)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    # a quarter of 0.5 and 2 within the factor's fp32 rounding: exact in bf16
    assert g[-1] == 0.5 and g[0] == 0.125 and g[2 ** 31] == 0.125
    assert (g[:-1] == 0.125).all()


def test_clipped_in_a_graph():
    grads = make([3000, 65, 12_345], "mixed")
    outs = [torch.empty_like(g) for g in grads]
    S.clip_grad_norm(grads, 1.0, out=outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = S.clip_grad_norm(grads, 1.0, out=outs)
    for seed in (1, 2, 3):
        for g, n in zip(grads, make([3000, 65, 12_345], "mixed", seed=seed, std=seed)):
            g.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        check(grads, outs, norm, 1.0)
        eager = [torch.empty_like(g) for g in grads]
        S.clip_grad_norm(grads, 1.0, out=eager)
        for a, b in zip(eager, outs):
            assert torch.equal(a, b)


def test_version_counters_move():
    """Autograd notices that a saved tensor was clipped in place."""
    p = torch.ones(4, device="cuda", requires_grad=True)
    y = p * 2
    z = (y * y).sum()
    with torch.no_grad():
        S.clip_grad_norm([y.detach()], 0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
