"""The plain forms of the speculative-decoding operators against what they must satisfy."""
import numpy as np
import pytest
import torch

from oracle import speculative as sp


def test_emitted_tokens_are_distributed_as_the_target():
    # exact integration over u and s for one draft: P(token = x) = sum over drafts d of
    # q(d) [min(1, p/q)(d) 1(x = d) + (1 - min(1, p/q)(d)) rest(x)], which must be p(x); checked
    # here by running the oracle on a fine grid of (d, u, s)
    p = torch.tensor([0.5, 0.25, 0.125, 0.125])
    q = torch.tensor([0.125, 0.5, 0.25, 0.125])
    grid = 64
    mass = np.zeros(4)
    for d in range(4):
        for i in range(grid):
            u = (i + 0.5) / grid
            for j in range(grid):
                s = (j + 0.5) / grid
                t, a = sp.verify_drafts(torch.stack([p, p])[None], q[None, None], torch.tensor([[d]]),
                                        torch.tensor([[u]]), torch.tensor([s]))
                mass[t[0, 0]] += float(q[d]) / grid ** 2
    assert np.abs(mass - p.numpy()).max() <= 1e-12   # the grid is aligned with the quarters


@pytest.mark.parametrize("s,want", [(0.0, 1), (0.24, 1), (0.25, 3), (0.999, 3), (1.5, 3), (-1.0, 1), (float("nan"), 1)])
def test_the_draw_takes_the_first_sum_above_the_number(s, want):
    p = torch.tensor([[[0.0, 0.25, 0.0, 0.75, 0.0]]])
    t, a = sp.verify_drafts(p, None, torch.zeros(1, 0), torch.zeros(1, 0), torch.tensor([s]))
    assert t.tolist() == [[want]] and a.tolist() == [0]


def test_nothing_left_draws_from_the_target_and_an_empty_row_gives_none():
    p = torch.tensor([[[0.5, 0.5], [0.0, 0.0]]])
    t, a = sp.verify_drafts(p, p[:, :1], torch.tensor([[0]]), torch.tensor([[1.0]]), torch.tensor([0.75]))
    assert t.tolist() == [[1, -1]] and a.tolist() == [0]   # u q = p: rejected, p - q is zero
    t, a = sp.verify_drafts(p, None, torch.tensor([[1]]), torch.tensor([[0.0]]), torch.tensor([0.5]))
    assert t.tolist() == [[1, -1]] and a.tolist() == [1]


def test_commit_then_step_is_the_recurrence():
    gen = torch.Generator().manual_seed(3)
    import oracle
    T, c = 5, 3
    q, k, v = (torch.randn(T + c, 1, 128, generator=gen).to(torch.bfloat16) for _ in range(3))
    g = -torch.rand(T + c, 1, generator=gen)
    S0 = torch.randn(1, 1, 128, 128, generator=gen)
    Q, K, V, G = (t[:, 0].double().numpy() for t in (q, k, v, g))
    o, kept = sp.draft_step(Q[c:], K[c:], V[c:], G[c:], 0.125, S0[0, 0].numpy(), (K, V, G), c)
    cu = torch.tensor([0, T + c])
    ref, hT = oracle.recurrent(q, k, v, g, 0.125, h0=S0, cu_seqlens=cu)
    assert np.abs(o - np.asarray(ref).reshape(T + c, 128)[c:]).max() <= 1e-12
    _, h = oracle.recurrent(q[:c], k[:c], v[:c], g[:c], 0.125, h0=S0, cu_seqlens=torch.tensor([0, c]))
    assert np.abs(kept - np.asarray(h).reshape(128, 128)).max() <= 1e-12


def test_fork_and_compact_lists():
    assert sp.fork([1, 0, 1, 0, 0], [2, -2, -1, 1, 0, 0]) == ([1, -1, 3, -1, 4, -1], [1, 1, 1, 1, 1])
    moves, mapping, m = sp.compact([0, 1, 0, 1, 1, 0])
    assert (moves, mapping, m) == ([(3, 0), (4, 2)], [-1, 1, -1, 0, 2, -1], 3)
