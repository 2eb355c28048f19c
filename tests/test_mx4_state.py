"""States of Mx4Linear: one of another number of columns does not load, on the CPU."""
import io

import pytest
import torch

import unstructured_sparse_linear_amd as P
from test_module_casts import linear


def saved(m, how):
    state = m.state_dict()
    if how == "file":
        f = io.BytesIO()
        torch.save(state, f)
        f.seek(0)
        state = torch.load(f, weights_only=True)
    return state


@pytest.mark.parametrize("how", ["object", "file"])
@pytest.mark.parametrize("nested", [False, True])
def test_a_state_of_other_columns_is_refused(how, nested):
    """70 and 96 columns have the same number of blocks."""
    def model(*args):
        m = linear(*args)
        return torch.nn.Sequential(torch.nn.ReLU(), m) if nested else m

    for a, b in ((96, 70), (70, 96), (33, 64)):
        m = model(b)
        want = {k: v.clone() for k, v in m.state_dict().items()}
        with pytest.raises(RuntimeError, match=f"{a} columns.*{b}"):
            m.load_state_dict(saved(model(a, 5, 1), how))
        assert all(torch.equal(v, want[k]) for k, v in m.state_dict().items())
        other = model(b, 5, 2)
        m.load_state_dict(saved(other, how))
        assert all(torch.equal(v, m.state_dict()[k]) for k, v in other.state_dict().items())
        assert sorted(k.split(".")[-1] for k in m.state_dict()) == ["codes", "scales"]


def test_a_state_without_its_columns():
    """A plain dict, as from a file that holds tensors alone: codes past the last column
    show that it was wider; others load."""
    m = linear(70)
    with pytest.raises(RuntimeError, match="past column 70"):
        m.load_state_dict(dict(linear(96, 5, 1).state_dict()))
    other = linear(70, 5, 2)
    m.load_state_dict(dict(other.state_dict()))
    assert torch.equal(m.codes, other.codes)
    # an odd last column: its byte's other half
    m = linear(69)
    with pytest.raises(RuntimeError, match="past column 69"):
        m.load_state_dict(dict(linear(70, 5, 1).state_dict()))
    m.load_state_dict(dict(linear(69, 5, 1).state_dict()))
    with pytest.raises(RuntimeError, match="Missing"):
        m.load_state_dict({})
    with pytest.raises(RuntimeError, match="size mismatch"):
        m.load_state_dict(dict(linear(300).state_dict()))
    assert not m.load_state_dict({}, strict=False).unexpected_keys
