"""Positions over several rounds of speculation in a layer with the q/k prologue (RMSNorm with a weight,
RoPE): each round normalises and rotates the raw q and k of its tokens in place with sala_gla_qk_prologue,
the first of them at the number of tokens kept so far, and after rejections the next round starts that
much earlier. Every kept token's output, and the states at the end, against the pooled one-token step with
the prologue in its kernel, token by token over the kept tokens alone.

The two paths round q and k to bf16 at the same place, after the same fp32 arithmetic in another order, so
an element may differ by a step of bf16, 2^-7 of it, here and there; outputs and states are compared as the
fused prologue is with the oracle (relative Frobenius error 1e-2 and 5e-3)."""
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
N, H, P, K, ROUNDS, SCALE = 5, 3, 8, 4, 6, 128 ** -0.5


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_linear_attention_gb300 import build, sala_gla
    build.build()
    return sala_gla


def test_positions_after_rejections(sg):
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    weights = [(1 + 0.1 * rand(128)).to(torch.bfloat16) for _ in range(2)]
    slots = torch.tensor([6, 0, 3, 7, 2], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 5, 900, 31000, 64], dtype=torch.int64, device="cuda")
    first = 0.3 * rand(P, H, 128, 128)
    pool, ref = first.clone(), first.clone()
    pos, pending, accepted, ref_pos = start.clone(), None, None, start.clone()
    for r in range(ROUNDS):
        q, k, v = ((3 * rand(N, K + 1, H, 128)).to(torch.bfloat16) for _ in range(3))
        g = torch.nn.functional.logsigmoid(2 + rand(N, K + 1, H))
        q2, k2 = q.clone(), k.clone()
        sg.qk_prologue(q2, k2, *weights, start_pos=pos)
        o = sg.recurrent_draft_step(q2, k2, v, g, SCALE, pool, slots, pending=pending, accepted=accepted)
        # what a verification says: every number of accepted drafts comes up
        accepted = ((torch.arange(N, device="cuda") + r) % (K + 1)).to(torch.int32)
        pending = (k2, v, g)
        pos = pos + accepted + 1
        for t in range(K + 1):
            kept = accepted >= t
            want = sg.recurrent_step_indexed(q[:, t].contiguous(), k[:, t].contiguous(), v[:, t].contiguous(), g[:, t].contiguous(),
                                             SCALE, ref, torch.where(kept, slots, -1).to(torch.int32),
                                             prologue=(*weights, 1e-6, 10000.0), positions=ref_pos)
            ref_pos = ref_pos + kept
            if kept.any():
                assert oracle.rel_fro(o[kept, t].float().cpu(), want[kept].double().cpu().numpy()) <= 1e-2
        assert torch.equal(pos, ref_pos)
    sg.recurrent_draft_step(None, None, None, None, SCALE, pool, slots, pending=pending, accepted=accepted)
    assert sg.get_device_status() == 0
    at = slots.long()
    assert oracle.rel_fro(pool[at].cpu(), ref[at].double().cpu().numpy()) <= 5e-3
    assert float((pos - start).min()) >= ROUNDS
