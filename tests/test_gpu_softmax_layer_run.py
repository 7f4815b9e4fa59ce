"""The softmax layers' operators together, as a server runs them: prompts in chunks, decoding and drafted tokens over a
cache that evicts back to a budget, and scores of the answer. Every step against the plain form on the same cache.

A step's attention is checked with the bounds that tests/test_gpu_paged_attention.py derives. The plain cache then takes the
library's weights, so that both evict by the same numbers: near ties would otherwise fall either way."""
import math

import pytest
import torch

from paged_inputs import bits, on_cpu, on_gpu

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
N, HQ, H, PAGE, BUDGET = 4, 32, 2, 16, 96


def _cache(kind):
    gen = torch.Generator().manual_seed(11)
    width = 12
    P = N * width
    c = dict(table=torch.randperm(P, generator=gen).to(torch.int32).reshape(N, width), lens=torch.zeros(N, dtype=torch.int32),
             k_scale=None, v_scale=None, weights=torch.full((P, H, PAGE), math.nan))
    dt = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    c["k_pages"], c["v_pages"] = (torch.full((P, H, PAGE, 128), math.nan).to(dt) for _ in range(2))
    if kind == "e4m3":
        c["k_scale"], c["v_scale"] = torch.tensor([0.02, 0.03]), torch.tensor([0.015, 0.01])
    return c


def _step(lib, g, r, gen, counts):
    """Appends and attends `counts` new tokens of each request; returns the outputs."""
    from oracle import softmax_layers as ref
    T = sum(counts)
    cu = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0)
    qkv = torch.randn(T, HQ + 2 * H, 128, generator=gen).to(torch.bfloat16)
    q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + H], qkv[:, HQ + H:]
    d, dcu = qkv.cuda(), cu.cuda()
    g.kv_lens += torch.tensor(counts, dtype=torch.int32, device="cuda")
    r.lens = [a + b for a, b in zip(r.lens, counts)]
    lib.kv_append(g, d[:, HQ:HQ + H], d[:, HQ + H:], cu_seqlens=dcu)
    o, lse = lib.paged_attention(d[:, :HQ], g, SCALE, cu_seqlens=dcu, accumulate=True)
    ref.append(r, k, v, cu)
    ro, rlse, (mass, size) = ref.attend(r, q, SCALE, cu, accumulate=True)
    E = 128 * 2.0 ** -24 * size + 2.0 ** -21 + 130 * 2.0 ** -24
    assert bool(((lse.cpu().double() - rlse).abs() <= E + 2.0 ** -22 * rlse.abs()).all())
    err, bound = (o.cpu().double() - ro).abs(), (2.0 ** -8 + 2 * E[..., None] + 2.0 ** -16) * mass + 2.0 ** -8 * ro.abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    for n, end in enumerate(r.lens):      # weights of every cached token, then the library's for both
        for i in range(end):
            page, slot = r.slot(n, i)
            got = g.weights[page, :, slot].cpu().double()
            assert bool(((got - r.w[page, :, slot]).abs() <= 1e-5 * r.w[page, :, slot] + 1e-9).all())
            r.w[page, :, slot] = got
    return o


def _evict(lib, g, r):
    from oracle import softmax_layers as ref
    lens, kept = lib.kv_evict(g, BUDGET, sinks=4, recent=24)
    want, places = ref.evict(r, BUDGET, 4, 24)
    assert torch.equal(kept.cpu(), places) and torch.equal(lens.cpu(), want)
    g.kv_lens.copy_(lens)
    r.lens = want.tolist()
    for n, end in enumerate(r.lens):
        for i in range(end):
            page, slot = r.slot(n, i)
            assert torch.equal(g.k_pages[page, :, slot].cpu().float().double(), r.k[page, :, slot])
            assert torch.equal(g.v_pages[page, :, slot].cpu().float().double(), r.v[page, :, slot])
            assert torch.equal(g.weights[page, :, slot].cpu().double(), r.w[page, :, slot])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prompts_decoding_drafts_and_eviction(kind):
    from gated_linear_attention_gb300 import sala_gla as lib
    from oracle import softmax_layers as ref
    c = _cache(kind)
    g, r, gen = on_gpu(c), on_cpu(c), torch.Generator().manual_seed(3)
    for counts in ([70, 33, 0, 1], [60, 40, 90, 0]):      # prompts in chunks, one request later
        _step(lib, g, r, gen, counts)
    _evict(lib, g, r)
    for counts in ([1, 1, 1, 1], [5, 1, 5, 0], [1, 30, 1, 1]):
        o = _step(lib, g, r, gen, counts)
        _evict(lib, g, r)
    # the answer's scores, from a small head
    head = torch.randn(HQ * 128, 1000, generator=gen, dtype=torch.float32) / 32
    logits = (o.reshape(o.shape[0], -1).float() @ head.cuda())
    tokens = torch.randint(0, 1000, (o.shape[0],), generator=gen, dtype=torch.int32)
    lp, ent, ids, vals = lib.token_logprobs(logits, tokens.cuda(), top=5)
    want = ref.logprobs(logits, tokens, 5)
    assert torch.equal(ids.cpu(), want[2])
    for a, b in ((lp, want[0]), (ent, want[1]), (vals, want[3])):
        assert float((a.cpu().double() - b).abs().max()) <= 2e-5
    assert lib.get_device_status() == 0


def test_a_captured_step_serves_growing_requests():
    """One graph of append, attention and eviction, replayed while the lengths on the device change."""
    from gated_linear_attention_gb300 import sala_gla as lib
    c = _cache("bf16")
    g, e, gen = on_gpu(c), on_gpu(c), torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(N, 1, h, 128, generator=gen).to(torch.bfloat16).cuda() for h in (HQ, H, H))
    new = torch.zeros(N, dtype=torch.int32, device="cuda")

    def step(cache):
        lib.kv_append(cache, k, v)
        o, lse = lib.paged_attention(q, cache, SCALE, accumulate=True)
        lens, _ = lib.kv_evict(cache, 12, sinks=1, recent=3)
        return o, lse, lens

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg, ng = step(g)
    for i in range(30):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen).to(torch.bfloat16))
        new.copy_(torch.tensor([1, i % 2, 1, int(i > 7)], dtype=torch.int32))   # 0: a request that waits
        for cache in (g, e):
            cache.kv_lens += new
        graph.replay()
        oe, le, ne = step(e)
        assert torch.equal(og, oe) and torch.equal(lg, le) and torch.equal(ng, ne)
        g.kv_lens.copy_(ng)
        e.kv_lens.copy_(ne)
    assert torch.equal(g.kv_lens.cpu(), torch.tensor([12, 12, 12, 12], dtype=torch.int32)) and lib.get_device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_calls_in_a_row_read_what_the_call_before_wrote(kind):
    """Calls that start while the one before them ends: evictions that write the lengths which the next calls go by, from
    one buffer into the other, give the same bits as the same calls with the device idle between them."""
    from gated_linear_attention_gb300 import sala_gla as lib
    c = _cache(kind)
    gen = torch.Generator().manual_seed(8)
    for name in ("k_pages", "v_pages"):
        c[name] = torch.randn(c[name].shape, generator=gen).to(c[name].dtype)
    c["weights"] = torch.rand(c["weights"].shape, generator=gen)
    c["lens"] = torch.tensor([190, 130, 70, 192], dtype=torch.int32)
    q, k, v = (torch.randn(N, 3, h, 128, generator=gen).to(torch.bfloat16).cuda() for h in (HQ, H, H))

    def chain(wait):
        a = on_gpu(c)
        b = a.with_requests(a.block_table, torch.zeros_like(a.kv_lens))
        kept = torch.zeros(N, H, 176, dtype=torch.int32, device="cuda")
        out = []
        for i, budget in enumerate(range(176, 16, -16)):
            now, after = (a, b) if i % 2 == 0 else (b, a)
            for call in (lambda: lib.kv_append(now, k, v), lambda: lib.paged_attention(q, now, SCALE, accumulate=True),
                         lambda: lib.kv_evict(now, budget, sinks=2, recent=5, new_lens=after.kv_lens,
                                              kept=kept.view(-1)[:N * H * budget].view(N, H, budget))):
                out.append(call())
                if wait:
                    torch.cuda.synchronize()
            out.append(now.kv_lens)
        torch.cuda.synchronize()
        return [t for r in out if r is not None for t in (r if isinstance(r, tuple) else (r,)) if t.dtype != torch.int32] + \
               [a.kv_lens, b.kv_lens, kept, bits(a.k_pages), bits(a.v_pages), a.weights]

    want = chain(True)
    for _ in range(10):
        assert all(torch.equal(x, y) for x, y in zip(chain(False), want))
    assert lib.get_device_status() == 0
