"""A cache object whose tensors are replaced: the calls go by the new ones, what does not fit is refused and changes nothing."""
import pytest
import torch

from paged_inputs import make_cache, new_tokens, on_gpu

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def _attend(cache, q, **kw):
    from gated_linear_attention_gb300 import sala_gla
    return sala_gla.paged_attention(q, cache, SCALE, **kw)


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_assigned_tensors_are_used():
    from gated_linear_attention_gb300 import sala_gla
    c = make_cache([90, 300], 16, 2, seed=1, weights=True)
    q = new_tokens([6], 8, size=2.0)[0].reshape(2, 3, 8, 128).cuda()
    g = on_gpu(c)
    lens, _ = sala_gla.kv_evict(g, 64, sinks=2, recent=8)
    want = _attend(g.with_requests(g.block_table, lens), q)
    g.kv_lens = lens
    assert g.kv_lens is lens and _same(_attend(g, q), want)
    table = torch.cat([g.block_table.flip(0), torch.full((2, 3), -1, dtype=torch.int32, device="cuda")], 1)
    want = _attend(g.with_requests(table, lens), q)
    g.block_table = table
    assert _same(_attend(g, q), want)
    k, v = g.v_pages.clone(), g.k_pages.clone()
    want = _attend(sala_gla.KvCache(k, v, table, lens, weights=g.weights), q)
    g.k_pages, g.v_pages = k, v
    assert _same(_attend(g, q), want)
    g.weights = torch.zeros_like(g.weights)
    _attend(g, q, accumulate=True)
    assert abs(float(g.weights.sum()) - 2 * 3 * 8) < 1e-3
    g.weights = None
    with pytest.raises(ValueError):
        _attend(g, q, accumulate=True)
    e = on_gpu(make_cache([90, 300], 16, 2, "e4m3", seed=1))
    before, was = _attend(e, q), e.v_scale
    e.v_scale = was * 2
    assert torch.equal(_attend(e, q)[0], before[0] * 2)
    assert sala_gla.get_device_status() == 0


def test_lengths_changed_in_place():
    g = on_gpu(make_cache([90, 300], 16, 2, seed=1))
    q = new_tokens([2], 8)[0].reshape(2, 1, 8, 128).cuda()
    held = g.kv_lens
    g.kv_lens -= 20
    assert g.kv_lens is held
    shorter = torch.tensor([70, 280], dtype=torch.int32, device="cuda")
    assert _same(_attend(g, q), _attend(g.with_requests(g.block_table, shorter), q))


def test_what_does_not_fit_is_refused():
    g = on_gpu(make_cache([90, 300], 16, 2, seed=1, weights=True))
    q = new_tokens([2], 8)[0].reshape(2, 1, 8, 128).cuda()
    want = _attend(g, q)
    for name, value, err in (("kv_lens", g.kv_lens.long(), TypeError), ("kv_lens", g.kv_lens[:1], ValueError),
                             ("kv_lens", g.kv_lens.cpu(), ValueError), ("kv_lens", None, TypeError),
                             ("block_table", g.block_table[:1], ValueError), ("block_table", g.block_table.long(), TypeError),
                             ("k_pages", g.k_pages[:1], ValueError), ("v_pages", g.v_pages.float(), TypeError),
                             ("weights", g.weights[..., :8], ValueError), ("k_scale", torch.ones(2, device="cuda"), ValueError),
                             ("N", 3, AttributeError), ("H", 3, AttributeError), ("lens", g.kv_lens, AttributeError)):
        with pytest.raises(err):
            setattr(g, name, value)
    assert _same(_attend(g, q), want)
