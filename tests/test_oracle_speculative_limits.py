"""The oracle of the verification at the ends of its range, worked out by hand."""
import pytest
import torch

from oracle import speculative as sp


@pytest.mark.parametrize("s", [0.0, 0.5, 0.75, 1.0 - 2.0 ** -24])
def test_the_largest_sum(s):
    V = 1 << 20   # 2^63 units in all
    t, a = sp.verify_drafts(torch.ones(1, 1, V), None, torch.zeros(1, 0), torch.zeros(1, 0), torch.tensor([s]))
    assert t.tolist() == [[int(s * V)]] and a.tolist() == [0]
