"""Scores of batches with more parts of rows than warps, so that a warp goes through several, against torch in 64 bits.

Bounds: a lane's chain has at most V / 32 + 8 terms (a row in one part), the joins of lanes and parts at most 140; each term and each sum
2^-24. A lane's maximum moves at most once in 16 of its elements, V / 512 times, each 2^-21 (exp and products). So lse - m is off
by at most t = (V / 32 + 150) 2^-24 + V / 512 2^-21 + 2^-21, a log probability by that and 2^-22 of itself, and the entropy, whose
second sum has terms of at most e^d |d|, by t (2 + |entropy| + log V) and its roundings, 2^-22 of that."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("top", [0, 1, 20, 64])
@pytest.mark.parametrize("N,V", [(5501, 333), (9750, 65), (5000, 1999), (301, 50021), (1999, 20011)])
def test_more_parts_than_warps(dtype, top, N, V):
    from gated_linear_attention_gb300 import sala_gla
    gen = torch.Generator(device="cuda").manual_seed(N + top)
    x = (3 * torch.randn(N, V, generator=gen, device="cuda")).to(dtype)
    # rows of their own sort among the others: a maximum at either end, all alike, all but one masked
    x[::7, 0] = 30.0
    x[1::7, -1] = 30.0
    x[2::7] = 0.5
    x[3::7] = -math.inf
    x[3::7, V // 2] = 1.0
    tokens = torch.randint(0, V, (N, 2), generator=gen, device="cuda", dtype=torch.int32)
    lp, ent, ids, values = sala_gla.token_logprobs(x, tokens, top=top)
    assert sala_gla.get_device_status() == 0
    t = (V / 32 + 150) * 2.0 ** -24 + V / 512 * 2.0 ** -21 + 2.0 ** -21
    for n in range(0, N, 512):            # 64 bits, some rows at a time
        rows = slice(n, n + 512)
        want = x[rows].double().log_softmax(1)
        logp = want.gather(1, tokens[rows].long())
        fin = logp.isfinite()
        assert torch.equal(lp[rows][~fin].double(), logp[~fin])
        assert bool(((lp[rows].double() - logp)[fin].abs() <= t + 2.0 ** -22 * logp[fin].abs()).all())
        e = -torch.where(want.isfinite(), want.exp() * want, torch.zeros_like(want)).sum(1)
        assert bool(((ent[rows].double() - e).abs() <= (t + 2.0 ** -22) * (2 + e + math.log(V))).all())
        if top:
            order = x[rows].float().sort(dim=1, descending=True, stable=True)
            some = order.values[:, :top] > -math.inf
            assert torch.equal(ids[rows], torch.where(some, order.indices[:, :top], -1).to(torch.int32))
            best = want.gather(1, order.indices[:, :top])
            assert torch.equal(values[rows].isfinite(), some)
            assert bool(((values[rows].double() - best)[some].abs() <= t + 2.0 ** -22 * best[some].abs()).all())
