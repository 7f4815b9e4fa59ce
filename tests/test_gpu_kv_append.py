"""Appending to a paged cache against the plain form: bits of every page, untouched rows among them."""
import math

import pytest
import torch

from paged_inputs import bits, make_cache, new_tokens, on_cpu, on_gpu

pytestmark = pytest.mark.gpu


def _run(c, k, v, cu=None):
    from gated_linear_attention_gb300 import sala_gla
    from oracle import softmax_layers as ref
    g, r = on_gpu(c), on_cpu(c)
    sala_gla.kv_append(g, k.cuda(), v.cuda(), cu_seqlens=None if cu is None else cu.cuda())
    torch.cuda.synchronize()
    status = sala_gla.get_device_status()
    ref.append(r, k, v, cu)
    for got, want in ((g.k_pages, r.k), (g.v_pages, r.v)):
        got = got.cpu().to(torch.float32).double()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
    if g.weights is not None:
        assert torch.equal(g.weights.cpu().double(), r.w)
    return status


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H", [1, 2, 5])
def test_append_packed(kind, page, H):
    counts, lens = [3, 0, 17, 1, 40], [3, 20, 33, 300, 257]
    c = make_cache(lens, page, H, kind, seed=page + H, weights=True)
    k, cu = new_tokens(counts, H, 2)
    v, _ = new_tokens(counts, H, 3)
    assert _run(c, k, v, cu) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("N,T", [(1, 1), (3, 1), (2, 5), (1, 70)])
def test_append_equal_counts(kind, N, T):
    c = make_cache([T + 9 * n for n in range(N)], 16, 2, kind, seed=N)
    k, _ = new_tokens([N * T], 2, 4)
    v, _ = new_tokens([N * T], 2, 5)
    assert _run(c, k.reshape(N, T, 2, 128), v.reshape(N, T, 2, 128)) == 0


def test_append_places_and_rows_that_are_not_there():
    """More tokens than the length: the first have no place. Tokens behind the last request stay out."""
    c = make_cache([4, 0, 18], 16, 2)
    k, cu = new_tokens([7, 2, 3], 2)
    more = torch.cat([k, torch.full((5, 2, 128), 9.0, dtype=torch.bfloat16)])
    assert _run(c, more, more, cu) == 0


def test_append_values_of_every_kind():
    c = make_cache([6], 16, 2, "e4m3")
    k, cu = new_tokens([6], 2, size=3.0)
    k[0, 0, :8] = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, 1e30, -1e30, 1e-30])
    assert _run(c, k, -k, cu) == 0
    c = make_cache([6], 16, 2, "bf16")
    assert _run(c, k, -k, cu) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_slices_of_a_projection(kind):
    c = make_cache([9, 30], 16, 2, kind)
    qkv, cu = new_tokens([9, 4], 12)
    k, v = qkv[:, 8:10], qkv[:, 10:12]
    from gated_linear_attention_gb300 import sala_gla
    from oracle import softmax_layers as ref
    g, r, d = on_gpu(c), on_cpu(c), qkv.cuda()
    sala_gla.kv_append(g, d[:, 8:10], d[:, 10:12], cu_seqlens=cu.cuda())
    ref.append(r, k, v, cu)
    assert torch.equal(g.k_pages.cpu().float().double(), r.k) and torch.equal(g.v_pages.cpu().float().double(), r.v)


def test_append_bad_tables_lengths_and_offsets():
    from gated_linear_attention_gb300 import sala_gla
    for bad in (-1, 99, 2 ** 31 - 1, -2 ** 31):
        c = make_cache([20, 20], 16, 2)
        c["table"][1, 1] = bad
        g, before = on_gpu(c), c["k_pages"].clone()
        k, cu = new_tokens([2, 2], 2)
        sala_gla.kv_append(g, k.cuda(), k.cuda(), cu_seqlens=cu.cuda())
        assert sala_gla.get_device_status() == 8
        changed = (g.k_pages.cpu() != before).any(-1).any(1).nonzero().tolist()
        assert changed == [[int(c["table"][0, 1]), s] for s in (2, 3)]
    for lens in ([-1, 20], [33, 20]):
        c = make_cache([20, 20], 16, 2)
        c["lens"][0] = lens[0]
        g = on_gpu(c)
        k, cu = new_tokens([2, 2], 2)
        sala_gla.kv_append(g, k.cuda(), k.cuda(), cu_seqlens=cu.cuda())
        assert sala_gla.get_device_status() == 8
        assert int((g.k_pages.cpu() != c["k_pages"]).any(-1).any(1).sum()) == 2
    for cu in ([0, 3, 2], [0, -1, 4], [0, 2, 9], [5, 2, 4]):
        c = make_cache([20, 20], 16, 2)
        g = on_gpu(c)
        k, _ = new_tokens([4], 2)
        sala_gla.kv_append(g, k.cuda(), k.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int64).cuda())
        assert sala_gla.get_device_status() == 6


def test_append_on_another_stream_and_in_a_graph():
    from gated_linear_attention_gb300 import sala_gla
    c = make_cache([9, 30], 16, 2)
    k, cu = new_tokens([2, 1], 2)
    g0, g1, g2 = on_gpu(c), on_gpu(c), on_gpu(c)
    d, dcu = k.cuda(), cu.cuda()
    sala_gla.kv_append(g0, d, d, cu_seqlens=dcu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    sala_gla.kv_append(g1, d, d, cu_seqlens=dcu, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sala_gla.kv_append(g2, d, d, cu_seqlens=dcu)
    graph.replay()
    torch.cuda.synchronize()
    for g in (g1, g2):
        assert torch.equal(bits(g.k_pages), bits(g0.k_pages)) and torch.equal(bits(g.v_pages), bits(g0.v_pages))
