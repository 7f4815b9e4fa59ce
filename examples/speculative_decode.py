"""Speculative decoding on lightning layers: a small random model, a one-layer drafter, and the
library's calls as a server makes them.

    python examples/speculative_decode.py [--layers 4] [--heads 8] [--samples 8] [--drafts 4] [--tokens 64]

The prompt goes through the chunked prefill once; its states are forked for every sample
(state_pool_fork). Each round, the drafter runs ahead on a scratch copy of its states
(state_pool_copy, recurrent_step_indexed), the target runs [last token, drafts] in one call that
first commits what it accepted the round before (recurrent_draft_step), and verify_drafts keeps the
drafts that the target agrees with and draws the next token. Nothing is read back by the host until
the end. Finished samples are freed and the pool is compacted.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_linear_attention_gb300 import inputs, sala_gla as sg  # noqa: E402

D = 128


class Stack:
    """Embedding, lightning layers without MLPs, output projection; random weights."""

    def __init__(self, layers, heads, vocab, slots, seed, like=None, state=torch.bfloat16):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape):
            return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * shape[0] ** -0.5

        self.L, self.H, width = layers, heads, heads * D
        self.embedding = w(vocab, width) * vocab ** 0.5 if like is None else like.embedding
        self.head = w(width, vocab) if like is None else like.head
        self.qkv = [w(width, 3 * width) for _ in range(layers)]
        self.out = [w(width, width) for _ in range(layers)]
        self.gate = inputs.const_head_gate(heads).cuda()
        self.pool = torch.zeros(layers, slots, heads, D, D, dtype=state, device="cuda")

    def layer_inputs(self, layer, x):
        """q, k, v bf16 and g fp32 of x [..., width], heads split."""
        q, k, v = (x @ self.qkv[layer]).unflatten(-1, (3, self.H, D)).unbind(-3)
        q, k = (inputs.l2_normalise(t.float()).to(torch.bfloat16) for t in (q, k))
        return q, k, v.contiguous(), self.gate.expand(*x.shape[:-1], self.H).contiguous()

    def run(self, tokens, attend):
        """Logits (fp32) of tokens [..., T]; attend(layer, q, k, v, g) is the layer's attention."""
        x = self.embedding[tokens.long()]
        for layer in range(self.L):
            o = attend(layer, *self.layer_inputs(layer, x))
            x = x + 4.0 * o.flatten(-2) @ self.out[layer]
        x = inputs.rms_normalise(x.float()).to(torch.bfloat16)
        return 3.0 * (x @ self.head).float()

    def prefill(self, tokens, slot):
        """Logits of a prompt [1, T]; its final states go to `slot`."""
        def attend(layer, q, k, v, g):
            o, state = sg.chunk_fwd(q, k, v, g, inputs.SCALE)
            self.pool[layer, slot] = state[0].to(self.pool.dtype)
            return o
        return self.run(tokens, attend)

    def step(self, tokens, slots):
        """One token per sequence, states updated in place: logits [N, vocab]."""
        return self.run(tokens, lambda layer, q, k, v, g: sg.recurrent_step_indexed(
            q, k, v, g, inputs.SCALE, self.pool[layer], slots))

    def draft_step(self, tokens, slots, pending, accepted):
        """Tokens [N, T] after committing the accepted part of `pending`: logits, the next pending."""
        kept = []

        def attend(layer, q, k, v, g):
            kept.append((k, v, g))
            return sg.recurrent_draft_step(q, k, v, g, inputs.SCALE, self.pool[layer], slots,
                                           pending=pending[layer] if pending else None, accepted=accepted)
        return self.run(tokens, attend), kept

    def commit(self, slots, pending, accepted):
        for layer in range(self.L):
            sg.recurrent_draft_step(None, None, None, None, inputs.SCALE, self.pool[layer], slots,
                                    pending=pending[layer], accepted=accepted)


def distribution(logits, greedy):
    if not greedy:
        return logits.softmax(-1)
    return torch.nn.functional.one_hot(logits.argmax(-1), logits.shape[-1]).float()


def generate(target, drafter, prompt, samples, drafts, rounds, greedy=False, seed=0):
    """`rounds` rounds of speculative decoding of `samples` continuations of prompt [1, T].
    Returns (tokens [samples, rounds * (drafts + 1)], -1 where nothing was emitted; accepted
    [rounds, samples]). The prompt's own slot 0 stays as a cached prefix."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    models = (target, drafter)
    used = [torch.zeros(m.pool.shape[1], dtype=torch.int32, device="cuda") for m in models]
    for u in used:
        u[0] = 1
    logits = target.prefill(prompt, 0)[:, -1]
    drafter.prefill(prompt, 0)
    last = distribution(logits, greedy).expand(samples, -1).multinomial(1, generator=gen).to(torch.int32)
    parents = torch.zeros(samples, dtype=torch.int32, device="cuda")
    slots = sg.state_pool_fork(target.pool, used[0], parents)
    own = sg.state_pool_fork(drafter.pool, used[1], parents)
    scratch = sg.state_pool_fork(drafter.pool, used[1], torch.full_like(parents, -1))

    pending, accepted, emitted, counts = None, None, [last], []
    for _ in range(rounds):
        # the drafter runs ahead on copies of its states
        sg.state_pool_copy(drafter.pool, drafter.pool, scratch, own)
        tokens, q = [last], []
        for _ in range(drafts):
            q.append(distribution(drafter.step(tokens[-1][:, 0], scratch), greedy))
            tokens.append(q[-1].multinomial(1, generator=gen).to(torch.int32))
        tokens = torch.cat(tokens, 1)
        # the target checks all of them; what it accepted last round is committed by the same call
        logits, pending = target.draft_step(tokens, slots, pending, accepted)
        u = torch.rand(samples, drafts + 1, generator=gen, device="cuda")
        out, accepted = sg.verify_drafts(distribution(logits, greedy), torch.stack(q, 1), tokens[:, 1:].contiguous(),
                                         u[:, 1:].contiguous(), u[:, 0].contiguous())
        # the drafter's own states take the accepted tokens
        _, kept = drafter.draft_step(tokens, own, None, None)
        drafter.commit(own, kept, accepted)
        last = out.gather(1, accepted[:, None].long())
        emitted.append(out)
        counts.append(accepted)
    target.commit(slots, pending, accepted)
    # all samples end: their slots are free again, the cached prefix moves to the front
    sg.state_pool_free(used[0], slots)
    sg.state_pool_compact(target.pool, used[0])
    return torch.cat(emitted, 1), torch.stack(counts)


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("layers", 4), ("heads", 8), ("vocab", 4096), ("samples", 8), ("drafts", 4), ("tokens", 64),
                        ("prompt", 200)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--greedy", action="store_true")
    a = ap.parse_args()
    torch.cuda.set_device(0)
    target = Stack(a.layers, a.heads, a.vocab, 2 * a.samples + 2, seed=1)
    drafter = Stack(1, a.heads, a.vocab, 2 * a.samples + 2, seed=2, like=target)
    drafter.qkv[0], drafter.out[0] = target.qkv[0], target.out[0]   # the target's first layer drafts
    prompt = torch.randint(0, a.vocab, (1, a.prompt), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    rounds = -(-a.tokens // (a.drafts + 1))
    generate(target, drafter, prompt, a.samples, a.drafts, 2, a.greedy)
    torch.cuda.synchronize()
    t = time.perf_counter()
    tokens, accepted = generate(target, drafter, prompt, a.samples, a.drafts, rounds, a.greedy)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    n = int((tokens >= 0).sum())
    print(f"{n} tokens of {a.samples} samples in {rounds} rounds, {1e3 * t:.1f} ms; {accepted.float().mean():.2f} of "
          f"{a.drafts} drafts accepted a round; device status {sg.get_device_status()}")


if __name__ == "__main__":
    main()
