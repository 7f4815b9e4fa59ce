"""The example of speculative decoding: what it emits greedily is what the target model alone says.
Every emitted token is scored by the chunked prefill over all tokens before it; its logit must be
the largest up to the rounding of bf16 activations (the two paths round the outputs of different
kernels: 2^-8 each over the layers' sums; an eighth of the logits' standard deviation is allowed)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_linear_attention_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import speculative_decode
    return speculative_decode


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafts", [1, 4])
def test_greedy_speculation_emits_the_targets_tokens(ex, drafts, state):
    samples, rounds, vocab = 3, 6, 1000
    target = ex.Stack(3, 4, vocab, 8, seed=1, state=state)
    drafter = ex.Stack(1, 4, vocab, 8, seed=2, like=target, state=state)
    drafter.qkv[0], drafter.out[0] = target.qkv[0], target.out[0]
    prompt = torch.randint(0, vocab, (1, 70), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    tokens, accepted = ex.generate(target, drafter, prompt, samples, drafts, rounds, greedy=True)
    assert ex.sg.get_device_status() == 0
    assert accepted.shape == (rounds, samples) and int(accepted.min()) >= 0 and int(accepted.max()) <= drafts
    for row in tokens:
        row = row[row >= 0]
        assert row.numel() >= rounds + 1
        text = torch.cat([prompt[0], row.long()])[None]
        logits = target.run(text, lambda layer, q, k, v, g: ex.sg.chunk_fwd(q, k, v, g, ex.inputs.SCALE)[0])[0]
        said = logits[prompt.shape[1] - 1:-1]
        behind = said.max(-1).values - said.gather(1, row.long()[:, None])[:, 0]
        assert float(behind.max()) <= 0.125 * float(said.std())


def test_sampled_speculation_runs(ex):
    target = ex.Stack(2, 4, 500, 20, seed=4)
    drafter = ex.Stack(1, 4, 500, 20, seed=5, like=target)
    prompt = torch.randint(0, 500, (1, 33), device="cuda")
    tokens, accepted = ex.generate(target, drafter, prompt, 8, 3, 5, seed=7)
    assert ex.sg.get_device_status() == 0
    emitted = (tokens >= 0).sum(1)
    assert torch.equal(emitted, 1 + (accepted + 1).sum(0)) and int(tokens.max()) < 500
