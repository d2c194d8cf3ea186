"""Conditions.fork's checks and what it moves, on the CPU."""

import pytest

torch = pytest.importorskip("torch")


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_fork_moves_rows():
    from semi_ar_draft_round_amd.logits import Conditions
    c = Conditions(4, 6, biases=2, device="cpu")
    c.state.copy_(torch.arange(24).view(4, 6))
    c.bias.copy_(torch.arange(8).view(4, 2))
    c.frequency.copy_(torch.arange(4))
    state, bias = c.state.clone(), c.bias.clone()
    c.fork(i32(3, -1, -7, 4))
    assert torch.equal(c.state, torch.stack([state[3], torch.zeros_like(state[1]), state[2], state[3]]))
    assert torch.equal(c.bias, bias[[3, 1, 2, 3]]) and c.frequency.tolist() == [3, 1, 2, 3]


@pytest.mark.parametrize("parent", [i32(1), i32(0, 1, 2), i32(0, 1, 2, 3, 0), i32(0, 1, 2, 3).view(4, 1),
                                    torch.zeros(4), torch.zeros(4, dtype=torch.bool)])
def test_fork_refuses(parent):
    """One parent for all slots, too, which would be broadcast."""
    from semi_ar_draft_round_amd.logits import Conditions
    c = Conditions(4, 6, biases=2, device="cpu")
    c.state.copy_(torch.arange(24).view(4, 6))
    before = c.state.clone()
    with pytest.raises(ValueError, match="parent"):
        c.fork(parent)
    assert torch.equal(c.state, before)
