"""Calls of the C interface that leave out outputs (the binding always has them): the same pages, weights and results."""
import pytest
import torch

from paged_inputs import bits, make_cache, new_tokens, on_gpu

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,L", [(1, 2000), (5, 700), (40, 300)])
def test_attention_without_lse(kind, T, L):
    from gated_linear_attention_gb300 import sala_gla
    c = make_cache([L, 50], 32, 2, kind, seed=T, weights=True)
    q = new_tokens([2 * T], 8, size=2.0)[0].reshape(2, T, 8, 128).cuda()
    for accumulate in (0, 1):
        a, b = on_gpu(c), on_gpu(c)
        want, _ = sala_gla.paged_attention(q, a, SCALE, accumulate=bool(accumulate))
        o = torch.empty_like(want)
        rc = sala_gla.load().sala_gla_paged_attention(b._ref, q.data_ptr(), 8 * 128, SCALE, None, o.data_ptr(), None, accumulate, 2, T,
                                                      8, torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and sala_gla.get_device_status() == 0
        assert torch.equal(o, want) and torch.equal(a.weights, b.weights)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("budget,sinks,recent", [(100, 4, 20), (1, 0, 0), (333, 0, 333), (5000, 3, 7), ((1 << 31) - 1, 4, 4)])
def test_eviction_without_kept_and_lengths(kind, budget, sinks, recent):
    from gated_linear_attention_gb300 import sala_gla
    c = make_cache([1500, 90, 0, 334], 64, 2, kind, seed=4, weights=True)
    a, b = on_gpu(c), on_gpu(c)
    sala_gla.kv_evict(a, min(budget, 5000), sinks=sinks, recent=recent)
    for lens in (torch.zeros(4, dtype=torch.int32, device="cuda"), None):
        b = on_gpu(c)
        rc = sala_gla.load().sala_gla_kv_evict(b._ref, budget, sinks, recent, None if lens is None else lens.data_ptr(), None, 4,
                                               torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and sala_gla.get_device_status() == 0
        assert lens is None or lens.tolist() == [min(x, budget) for x in (1500, 90, 0, 334)]
        for x, y in ((a.k_pages, b.k_pages), (a.v_pages, b.v_pages), (a.weights, b.weights)):
            assert torch.equal(bits(x), bits(y))
