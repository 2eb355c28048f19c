"""Low-rank adapters whose output shares memory with their input: a square
layer's residual in place, rows shifted by some, and neighbouring columns."""
import pytest
import torch

import unstructured_sparse_linear_amd as S
import lowrank_ref as ref

pytestmark = pytest.mark.gpu
N = 320


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    S.lib()
    yield
    torch.cuda.synchronize()


def case(dt, T, R=16):
    return ref.Case(dt, [T], [1], 2, R, N, N, seed=T)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 3, 16, 17])
def test_square_layer_in_place(dt, T):
    for R in (16, 20):
        c = case(dt, T, R)
        c.yt = c.xt
        want = ref.add(c)
        buf = c.xt.clone()
        c.xt = buf
        assert S.low_rank_add(buf, *c.args(), out=buf) is buf
        ref.check(buf, want, "yt, xt and out are one")
        again = case(dt, T, R)
        buf = again.xt
        S.low_rank_add(buf, *again.args(), out=buf)
        ref.check(buf, want, "the same again")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 16, 17])
@pytest.mark.parametrize("call", ["add", "project"])
def test_out_over_xt(dt, T, call):
    for shift in (0, 7, -7):
        c = case(dt, T)
        want = ref.add(c) if call == "add" else ref.project(c)
        room = torch.zeros(N + 14, T, dtype=c.xt.dtype, device="cuda")
        x, out = room[7:7 + N], room[7 + shift:7 + shift + N]
        x.copy_(c.xt)
        c.xt = x
        got = (S.low_rank_add(c.yt, *c.args(), out=out) if call == "add"
               else S.low_rank_project(c.W, *c.args(), out=out))
        assert got is out
        ref.check(out, want, f"rows shifted by {shift}")


@pytest.mark.parametrize("T", [1, 16])
def test_columns_of_one_buffer(T):
    """xt, yt and out lie between each other's rows and share no value."""
    c = case("bf16", T)
    room = torch.zeros(N, 3 * T, dtype=torch.bfloat16, device="cuda")
    x, y, out = room[:, :T], room[:, T:2 * T], room[:, 2 * T:]
    x.copy_(c.xt)
    y.copy_(c.yt)
    kept = room[:, :2 * T].clone()
    c.xt = x
    S.low_rank_add(y, *c.args(), out=out)
    ref.check(out, ref.add(c))
    S.low_rank_project(c.W, *c.args(), out=out)
    ref.check(out, ref.project(c))
    assert torch.equal(room[:, :2 * T], kept)
