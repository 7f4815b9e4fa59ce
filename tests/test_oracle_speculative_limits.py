"""The oracle of the verification at the ends of its range, worked out by hand."""
import pytest
import torch

from oracle import speculative as sp


@pytest.mark.parametrize("s", [0.0, 0.5, 0.75, 1.0 - 2.0 ** -24])
def test_the_largest_sum(s):
    V = 1 << 20   # 2^63 units in all
    t, a = sp.verify_drafts(torch.ones(1, 1, V), None, torch.zeros(1, 0), torch.zeros(1, 0), torch.tensor([s]))
    assert t.tolist() == [[int(s * V)]] and a.tolist() == [0]


@pytest.mark.parametrize("p,q,u,ok", [(0.0, -1.0, 0.5, False), (0.25, float("nan"), 0.5, True), (float("nan"), 0.5, 0.0, False),
                                      (0.75, 2.0, 0.5, True), (2.0, 1.5, 1.0, False), (0.5, 0.5, 0.5, True)])
def test_the_accept_test_takes_values_as_probabilities(p, q, u, ok):
    P, Q = torch.zeros(1, 2, 5), torch.zeros(1, 1, 5)
    P[:, :, 3], P[0, 0, 1], Q[0, 0, 1] = 1.0, p, q
    assert sp.verify_drafts(P, Q, torch.tensor([[1]]), torch.tensor([[u]]), torch.zeros(1))[1].tolist() == [int(ok)]
