"""Eviction by accumulated weight against the plain form: every page, weight and kept place, bit for bit."""
import math

import pytest
import torch

from paged_inputs import bits, make_cache, on_cpu, on_gpu

pytestmark = pytest.mark.gpu


def _run(c, budget, sinks=0, recent=0):
    from gated_linear_attention_gb300 import sala_gla
    from oracle import softmax_layers as ref
    g, r = on_gpu(c), on_cpu(c)
    lens, kept = sala_gla.kv_evict(g, budget, sinks=sinks, recent=recent)
    status = sala_gla.get_device_status()
    want_lens, want_kept = ref.evict(r, budget, sinks, recent)
    assert torch.equal(lens.cpu(), want_lens)
    assert torch.equal(kept.cpu(), want_kept)
    for got, want in ((g.k_pages, r.k), (g.v_pages, r.v), (g.weights, r.w)):
        got = got.cpu().to(torch.float32).double()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
    assert torch.equal(g.kv_lens.cpu(), c["lens"])
    return status


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("H", [1, 2, 5])
@pytest.mark.parametrize("budget,sinks,recent", [(64, 4, 16), (100, 0, 0), (33, 0, 33), (40, 40, 0), (41, 20, 21), (1, 0, 0)])
def test_evict(kind, page, H, budget, sinks, recent):
    c = make_cache([0, 1, 33, 64, 65, 100, 300], page, H, kind, seed=budget + H, weights=True)
    assert _run(c, budget, sinks, recent) == 0


@pytest.mark.parametrize("budget", [17, 500, 1100, 2000])
def test_evict_long(budget):
    c = make_cache([2500, 1030], 64, 2, seed=budget, weights=True)
    assert _run(c, budget, 4, 13) == 0


def test_more_keys_than_are_cached():
    c = make_cache([20011], 256, 1, seed=3, weights=True)
    assert _run(c, 9000, 16, 1000) == 0


@pytest.mark.parametrize("case", ["equal", "zeros", "few", "values", "steps"])
def test_ties_and_values_of_every_kind(case):
    c = make_cache([1500, 90], 16, 2, seed=5, weights=True)
    w = c["weights"]
    if case == "equal":
        w.fill_(0.25)
    elif case == "zeros":
        w.zero_()
    elif case == "few":
        w.copy_((w * 4).floor())
    elif case == "values":
        w[::3] = math.nan
        w[1::5] = -1.0
        w[2::7] = math.inf
        w[3::11] = 1e-42
        w[4::13] = -0.0
    else:
        w.copy_(torch.ldexp(torch.ones_like(w), (torch.arange(w.numel()) % 200 - 100).reshape(w.shape)))
    assert _run(c, 700, 3, 5) == 0
    assert _run(c, 64, 0, 1) == 0


def test_budget_above_every_length_and_repeated():
    c = make_cache([30, 64], 16, 2, weights=True)
    assert _run(c, 4096) == 0
    from gated_linear_attention_gb300 import sala_gla
    c = make_cache([300, 260], 16, 2, weights=True, seed=9)
    a, b = on_gpu(c), on_gpu(c)
    x, y = sala_gla.kv_evict(a, 100, 4, 10), sala_gla.kv_evict(b, 100, 4, 10)
    assert torch.equal(x[1], y[1]) and torch.equal(bits(a.k_pages), bits(b.k_pages))
    once = bits(a.k_pages).clone()
    lens, kept = sala_gla.kv_evict(a.with_requests(a.block_table, x[0]), 100, 4, 10)
    assert torch.equal(bits(a.k_pages), once) and lens.tolist() == [100, 100]
    assert torch.equal(kept.cpu(), torch.arange(100, dtype=torch.int32).expand(2, 2, 100))


def test_bad_tables_and_lengths():
    from gated_linear_attention_gb300 import sala_gla
    for bad in (-1, 1000, 2 ** 31 - 1):
        c = make_cache([90, 90], 16, 2, weights=True)
        c["table"][0, 3] = bad
        g = on_gpu(c)
        sala_gla.kv_evict(g, 50, 2, 2)
        assert sala_gla.get_device_status() == 8
    c = make_cache([90, 90], 16, 2, weights=True)
    c["lens"][0] = 500
    g = on_gpu(c)
    lens, kept = sala_gla.kv_evict(g, 50, 2, 2)
    assert sala_gla.get_device_status() == 8
    assert lens.tolist() == [0, 50] and int(kept[0].max()) == -1


def test_stream_and_graph():
    from gated_linear_attention_gb300 import sala_gla
    c = make_cache([700, 400], 32, 2, weights=True)
    a, b, d = on_gpu(c), on_gpu(c), on_gpu(c)
    want = sala_gla.kv_evict(a, 100, 4, 10)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    other = sala_gla.kv_evict(b, 100, 4, 10, stream=s)
    s.synchronize()
    with torch.cuda.graph(graph):
        third = sala_gla.kv_evict(d, 100, 4, 10)
    graph.replay()
    torch.cuda.synchronize()
    for g, got in ((b, other), (d, third)):
        assert torch.equal(got[1], want[1]) and torch.equal(bits(g.k_pages), bits(a.k_pages))
        assert torch.equal(bits(g.v_pages), bits(a.v_pages)) and torch.equal(g.weights, a.weights)


def test_refusals():
    from gated_linear_attention_gb300 import sala_gla
    g = on_gpu(make_cache([90], 16, 2, weights=True))
    for kw in (dict(budget=0), dict(budget=-3), dict(budget=10, sinks=-1), dict(budget=10, recent=-1),
               dict(budget=10, sinks=6, recent=5)):
        with pytest.raises(sala_gla.SalaError):
            sala_gla.kv_evict(g, **kw)
    with pytest.raises(sala_gla.SalaError):
        sala_gla.kv_evict(g, 10, new_lens=g.kv_lens)
    with pytest.raises(ValueError):
        sala_gla.kv_evict(on_gpu(make_cache([90], 16, 2)), 10)
