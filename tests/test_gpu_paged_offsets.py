"""Caches whose pages lie past 2^31 elements and 2^32 bytes: the same results as with the first pages."""
import pytest
import torch

from paged_inputs import bits, make_cache, new_tokens, on_gpu

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_past_32_bits(kind):
    from gated_linear_attention_gb300 import sala_gla as lib
    c = make_cache([300, 41], 64, 2, kind, seed=3, weights=True)
    small = on_gpu(c)
    used = c["k_pages"].shape[0]
    P = (1 << 32) // (2 * 64 * 128) // (1 if kind == "e4m3" else 2) + 4 * used     # past 2^32 bytes
    big = {n: torch.empty((P, *c[n].shape[1:]), dtype=c[n].dtype, device="cuda") for n in ("k_pages", "v_pages", "weights")}
    for n, t in big.items():
        t[P - used:].copy_(c[n])
    table = torch.where(c["table"] >= 0, c["table"] + (P - used), c["table"])
    large = lib.KvCache(big["k_pages"], big["v_pages"], table.cuda(), c["lens"].cuda(), small.k_scale, small.v_scale,
                        big["weights"])
    k, cu = new_tokens([7, 2], 2, 5)
    q, _ = new_tokens([7, 2], 32, 6, size=2.0)
    out = []
    for cache in (small, large):
        lib.kv_append(cache, k.cuda(), -k.cuda(), cu_seqlens=cu.cuda())
        o, lse = lib.paged_attention(q.cuda(), cache, SCALE, cu_seqlens=cu.cuda(), accumulate=True)
        lens, kept = lib.kv_evict(cache, 100, sinks=3, recent=10)
        tail = cache.k_pages.shape[0] - used
        out.append([o, lse, lens, kept] + [t[tail:] for t in (cache.k_pages, cache.v_pages, cache.weights)])
    assert lib.get_device_status() == 0
    for a, b in zip(*out):
        assert torch.equal(bits(a), bits(b))
