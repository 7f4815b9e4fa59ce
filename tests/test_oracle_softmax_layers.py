"""The plain forms of the softmax layers' operators against torch's own functions and by hand (CPU)."""
import math

import torch

from oracle import softmax_layers as ref
from paged_inputs import make_cache, new_tokens, on_cpu


def test_attend_is_causal_attention():
    c = make_cache([37], 16, 2, seed=1, weights=True)
    q, _ = new_tokens([9], 6, size=2.0)
    cache = on_cpu(c)
    o, lse, _ = ref.attend(cache, q.reshape(1, 9, 6, 128), 0.1, accumulate=True)
    k, v = (torch.stack([cache.rows(p, s, 0, h, 37) for h in range(2)]).repeat_interleave(3, 0)
            for p, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    mask = torch.ones(9, 37, dtype=torch.bool).tril(28)
    want = torch.nn.functional.scaled_dot_product_attention(q.double().transpose(0, 1), k, v, attn_mask=mask, scale=0.1)
    assert float((o[0].transpose(0, 1) - want).abs().max()) < 1e-12
    s = 0.1 * q.double().transpose(0, 1) @ k.transpose(1, 2)
    assert float((lse[0].t() - s.masked_fill(~mask, -math.inf).logsumexp(-1)).abs().max()) < 1e-12
    # a row's weights sum to one: 9 tokens of 3 heads each on a key/value head
    assert abs(float((cache.w - c["weights"].double()).sum()) - 9 * 6) < 1e-9


def test_append_then_evict_by_hand():
    c = make_cache([5], 16, 1, weights=True)
    cache = on_cpu(c)
    k = torch.arange(5.0)[:, None, None].expand(5, 1, 128).to(torch.bfloat16)
    ref.append(cache, k, 10 * k, torch.tensor([0, 5]))
    page = int(c["table"][0, 0])
    assert cache.k[page, 0, :5, 0].tolist() == [0, 1, 2, 3, 4] and cache.w[page, 0, :5].tolist() == [0.0] * 5
    cache.w[page, 0, :5] = torch.tensor([0.1, 0.5, math.nan, 0.5, 0.2], dtype=torch.float64)
    lens, kept = ref.evict(cache, 3, 1, 1)
    assert lens.tolist() == [3] and kept.tolist() == [[[0, 1, 4]]]
    assert cache.k[page, 0, :5, 0].tolist() == [0, 1, 4, 3, 4] and cache.v[page, 0, :3, 7].tolist() == [0, 10, 40]


def test_logprobs_is_log_softmax():
    x = torch.randn(3, 40)
    lp, ent, ids, vals = ref.logprobs(x, torch.tensor([[3], [39], [-1]], dtype=torch.int32), 4)
    want = x.double().log_softmax(1)
    assert torch.allclose(lp[:2, 0], torch.stack([want[0, 3], want[1, 39]])) and float(lp[2, 0]) == 0.0
    assert torch.allclose(ent, torch.distributions.Categorical(logits=x.double()).entropy())
    assert torch.equal(ids.long(), want.topk(4).indices) and torch.allclose(vals, want.topk(4).values)
