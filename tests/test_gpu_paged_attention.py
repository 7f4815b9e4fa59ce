"""Attention of new tokens over a paged cache against the plain form in 64 bits.

Bounds, from the arithmetic: a score is a sum of 128 products in fp32, off by at most A = 128 * 2^-24 *
scale * sum |q k| (worst row: `size`); exp2 and its argument are good to 2^-21 relative; a row's sum of n
positive terms is taken in chains of at most 128 + n / 128 terms, 2^-24 each. So log sum exp is off by at
most E = A + 2^-21 + (128 + n / 128) 2^-24 and the rounding of the result, 2^-22 |lse|. The weights p are off by
2 E relative and are rounded to bf16 for the product with v (2^-8, half a step), whose sum keeps fp32:
o is off by (2^-8 + 2 E + 2^-16) sum |p v| and its own rounding 2^-8 |o|. The accumulated weights are sums
of p in fp32 over R rows: 2 E + 2^-21 + R 2^-24 relative, and the rounding of the running sum."""
import math

import pytest
import torch

from paged_inputs import bits, make_cache, new_tokens, on_cpu, on_gpu

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def _compare(got, want, c, g, r, rows, seen=None):
    (o, lse), (ro, rlse, (mass, size)) = got, want
    n = max(c["lens"].tolist() + [1])
    E = 128 * 2.0 ** -24 * size.nan_to_num(0.0) + 2.0 ** -21 + (128 + n / 128) * 2.0 ** -24
    o, lse = o.cpu().double(), lse.cpu().double()
    has = ~rlse.isnan()                   # rows of a request
    assert torch.equal(lse[has & rlse.isinf()], rlse[has & rlse.isinf()])
    fin = rlse.isfinite()
    err = (lse - rlse).abs()
    assert bool((err <= E + 2.0 ** -22 * rlse.abs())[fin].all()), float(err[fin].max())
    err, bound = (o - ro).abs(), (2.0 ** -8 + 2 * E[..., None] + 2.0 ** -16) * mass + 2.0 ** -8 * ro.abs() + 1e-30
    assert bool((err <= bound)[has].all()), float((err / bound)[has].max())
    if r.w is not None and rows:
        e = float(E.max())
        was = c["weights"].double()
        err, bound = (g.weights.cpu().double() - r.w).abs(), (2 * e + 2.0 ** -21 + rows * 2.0 ** -24) * (r.w - was) + 2.0 ** -24 * r.w
        assert bool((err <= bound).all()), float(err.max())
    return has


def _run(c, q, cu=None, accumulate=False, scale=SCALE):
    from gated_linear_attention_gb300 import sala_gla
    from oracle import softmax_layers as ref
    g, r = on_gpu(c), on_cpu(c)
    got = sala_gla.paged_attention(q.cuda(), g, scale, cu_seqlens=None if cu is None else cu.cuda(),
                                   accumulate=accumulate)
    torch.cuda.synchronize()
    assert sala_gla.get_device_status() == 0
    want = ref.attend(r, q, scale, cu, accumulate)
    rows = (q.shape[1] if cu is None else int(cu.diff().max())) * q.shape[-2] // c["k_pages"].shape[1]
    _compare(got, want, c, g, r, rows if accumulate else 0)
    if c["weights"] is not None and not accumulate:
        assert torch.equal(g.weights.cpu(), c["weights"])
    return g, got


HEADS = [(1, 1), (2, 1), (8, 8), (16, 4), (5, 1), (14, 2), (24, 2), (32, 2), (12, 4), (64, 1), (128, 1)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,H", HEADS)
def test_one_token_each(kind, Hq, H):
    lens = [1, 2, 15, 16, 17, 127, 128, 129, 0, 300, 513]
    c = make_cache(lens, 16, H, kind, seed=Hq, weights=True)
    q, _ = new_tokens([len(lens)], Hq, size=2.0)
    _run(c, q.reshape(len(lens), 1, Hq, 128), accumulate=Hq % 3 != 2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("accumulate", [False, True])
def test_ragged_chunks(kind, page, accumulate):
    """Decoding rows, drafts, prompts of their own, chunks behind a prefix, and nothing, in one batch."""
    lens, counts = [200, 131, 90, 0, 411, 258, 33], [1, 5, 90, 0, 40, 0, 33]
    c = make_cache(lens, page, 2, kind, seed=page, weights=True)
    q, cu = new_tokens(counts, 32, size=2.0)
    _run(c, q, cu, accumulate)


@pytest.mark.parametrize("Hq,H", [(1, 1), (8, 8), (6, 2), (14, 2), (40, 8), (128, 1)])
def test_chunks_of_other_head_layouts(Hq, H):
    lens, counts = [140, 70, 300], [140, 3, 31]
    c = make_cache(lens, 32, H, seed=Hq, weights=True)
    q, cu = new_tokens(counts, Hq, size=1.5)
    _run(c, q, cu, accumulate=True)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 33, 129])
def test_chunk_ends(T):
    """Chunks around the ends of row tiles and of the tiles of the cache."""
    for L in {T, T + 1, 127 + T, 128 + T, 129 + T}:
        c = make_cache([L], 16, 2, seed=T, weights=True)
        q, _ = new_tokens([T], 32, size=2.0)
        _run(c, q.reshape(1, T, 32, 128), accumulate=L % 2 == 0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_long_cache_split_over_many_blocks(kind):
    c = make_cache([9001, 40], 64, 1, kind, seed=2, weights=True)
    q, cu = new_tokens([3, 2], 4, size=2.0)
    _run(c, q, cu, accumulate=True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,Hq", [(1, 16), (3, 16), (1, 64), (40, 16)])
def test_more_tiles_than_blocks(kind, T, Hq):
    """Blocks that go through several units of one to seven tiles each, whole and shared."""
    lens = [T + (137 * n) % 830 for n in range(61)]
    c = make_cache(lens, 32, 8, kind, seed=T, weights=True)
    q, _ = new_tokens([T * len(lens)], Hq, size=2.0)
    _run(c, q.reshape(len(lens), T, Hq, 128), accumulate=True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 9])
def test_short_units_one_after_another(kind, T):
    """Blocks that go through a dozen units of mostly one tile, some of two or three: the softmax groups lead them in turn."""
    lens = [T + (29 * n) % 118 + (130 if n % 5 == 3 else 0) + (100 if n % 7 == 6 else 0) for n in range(230)]
    c = make_cache(lens, 32, 8, kind, seed=T, weights=True)
    q, _ = new_tokens([T * len(lens)], 16, size=3.0)
    _run(c, q.reshape(len(lens), T, 16, 128), accumulate=True)


def test_more_requests_than_a_block_scans():
    lens = [1 + (53 * n) % 300 for n in range(300)]
    c = make_cache(lens, 16, 2, seed=1, weights=True)
    counts = [n % 3 for n in range(300)]
    q, cu = new_tokens(counts, 8, size=2.0)
    _run(c, q, cu, accumulate=True)


def test_peaked_and_growing_scores():
    """Scores that rise along the cache (the maximum moves in every tile), and far apart ones."""
    c = make_cache([700], 16, 1, seed=3)
    q, _ = new_tokens([6], 4, size=1.0)
    ramp = torch.linspace(0, 12, 700)
    for i in range(700):
        p, s = int(c["table"][0, i // 16]), i % 16
        c["k_pages"][p, 0, s] = (ramp[i] * torch.ones(128)).to(torch.bfloat16)
    q = torch.ones_like(q)
    q[1] *= -1
    q[2] *= 8
    q[3] *= -8
    _run(c, q.reshape(1, 6, 4, 128))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_growing_scores_of_two_query_tiles(kind):
    """The same for units of two query tiles, and tokens whose maximum stays beside some whose maximum moves."""
    c = make_cache([900], 32, 1, kind, seed=5, weights=True)
    unit = 1.0 if kind == "bf16" else float(c["k_scale"][0])
    for i in range(900):
        p, s = int(c["table"][0, i // 32]), i % 32
        c["k_pages"][p, 0, s] = (torch.full((128,), 0.01 * i) / unit).clamp(max=448 if kind == "e4m3" else 1e9).to(
            c["k_pages"].dtype)   # a cast to e4m3 alone makes NaN of what is above
    q, _ = new_tokens([24 * 16], 1, size=0.05)
    q = q.reshape(1, 24, 16, 128)
    q[0, ::3] += 1
    q[0, 1::3, ::2] -= 1
    _run(c, q, accumulate=True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,H,lens,counts", [(32, 2, [70, 129, 5, 0], [20, 1, 5, 3]), (3, 1, [300, 17], [150, 17]),
                                              (2, 2, [40, 600], [1, 1])])
def test_unused_rows_and_entries_do_not_enter(kind, Hq, H, lens, counts):
    """NaN in unused rows of pages and in pages nobody has, and table entries past the lengths that are no
    pages: the same bits as with zeros and valid entries there."""
    from gated_linear_attention_gb300 import sala_gla
    out = []
    for stale, past in ((0.0, 0), (math.nan, -7), (math.nan, 2 ** 31 - 1)):
        c = make_cache(lens, 32, H, kind, seed=8, weights=True, width=40, stale=stale, past=past)
        q, cu = new_tokens(counts, Hq, size=2.0)
        g = on_gpu(c)
        o, lse = sala_gla.paged_attention(q.cuda(), g, SCALE, cu_seqlens=cu.cuda(), accumulate=True)
        assert sala_gla.get_device_status() == 0
        out.append((o, lse, g.weights))
        assert not bool(o.isnan().any()) and not bool(lse.isnan().any())
    for other in out[1:]:
        for a, b in zip(out[0], other):
            assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("Hq,H,T,L", [(32, 2, 21, 150), (4, 4, 200, 260), (2, 1, 5, 40), (16, 1, 3, 300), (128, 1, 3, 130)])
def test_bad_values_of_later_tokens(value, Hq, H, T, L):
    """A bad key or value among the new tokens reaches the tokens that see it and nobody else."""
    from gated_linear_attention_gb300 import sala_gla
    for which in ("v_pages", "k_pages"):
        c = make_cache([L], 16, H, seed=6)
        clean = {n: None if t is None else t.clone() for n, t in c.items()}
        at = L - T + T // 2                     # seen by the tokens from T // 2 on
        page, slot, d = int(c["table"][0, at // 16]), at % 16, 37
        c[which][page, 0, slot, d] = value
        q, _ = new_tokens([T], Hq, size=1.0)
        q = q.reshape(1, T, Hq, 128)
        bad, _ = sala_gla.paged_attention(q.cuda(), on_gpu(c), SCALE)
        good, _ = sala_gla.paged_attention(q.cuda(), on_gpu(clean), SCALE)
        bad, good, G = bad.cpu()[0], good.cpu()[0], Hq // H
        assert torch.equal(bits(bad[:T // 2]), bits(good[:T // 2]))            # before it
        assert torch.equal(bits(bad[:, G:]), bits(good[:, G:]))                # other heads
        hit = bad[T // 2:, :G]
        if which == "v_pages":
            assert not bool(hit[..., d].isfinite().any())
            rest = torch.arange(128) != d
            assert torch.equal(bits(hit[..., rest]), bits(good[T // 2:, :G][..., rest]))
        elif math.isnan(value):
            assert bool(hit.isnan().all())


def test_queries_of_a_projection_and_rows_behind_the_last_request():
    from gated_linear_attention_gb300 import sala_gla
    c = make_cache([40, 9], 16, 2, seed=4)
    qkv, cu = new_tokens([6, 2], 36, size=2.0)
    qkv = torch.cat([qkv, torch.full((3, 36, 128), math.nan, dtype=torch.bfloat16)])
    q = qkv[:, :32]
    g, dev = on_gpu(c), qkv.cuda()
    want = sala_gla.paged_attention(q[:8].contiguous().cuda(), g, SCALE, cu_seqlens=cu.cuda())
    o, lse = torch.full((11, 32, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((11, 32), 7.0, device="cuda")
    sala_gla.paged_attention(dev[:, :32], g, SCALE, cu_seqlens=cu.cuda(), o=o, lse=lse)
    assert torch.equal(o[:8], want[0]) and torch.equal(lse[:8], want[1])
    assert bool((o[8:] == 7).all()) and bool((lse[8:] == 7).all())
    # a gap before the first request
    cu2 = cu + 3
    q2 = torch.cat([torch.zeros(3, 32, 128, dtype=torch.bfloat16), q[:8]]).cuda()
    o.fill_(7.0)
    sala_gla.paged_attention(q2, g, SCALE, cu_seqlens=cu2.cuda(), o=o)
    assert torch.equal(o[3:], want[0]) and bool((o[:3] == 7).all())


def test_requests_that_share_pages():
    c = make_cache([100, 60], 16, 2, seed=5)
    c["table"][1, :3] = c["table"][0, :3]
    q, cu = new_tokens([3, 7], 32, size=2.0)
    _run(c, q, cu)


def test_repeats_streams_graphs_and_calls_at_once():
    from gated_linear_attention_gb300 import sala_gla
    c = make_cache([1500, 200, 77], 16, 2, seed=7, weights=True)
    q, cu = new_tokens([9, 40, 1], 32, size=2.0)
    d, dcu = q.cuda(), cu.cuda()
    caches = [on_gpu(c) for _ in range(6)]
    want = sala_gla.paged_attention(d, caches[0], SCALE, cu_seqlens=dcu, accumulate=True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [sala_gla.paged_attention(d, caches[1], SCALE, cu_seqlens=dcu, accumulate=True, stream=s1),
           sala_gla.paged_attention(d, caches[2], SCALE, cu_seqlens=dcu, accumulate=True, stream=s2)]
    s1.synchronize(), s2.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, cache in zip(graphs, caches[3:5]):
        with torch.cuda.graph(graph):
            got.append(sala_gla.paged_attention(d, cache, SCALE, cu_seqlens=dcu, accumulate=True))
    graphs[0].replay(), graphs[1].replay()
    torch.cuda.synchronize()
    for cache, (o, lse) in zip(caches[1:5], got):
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(cache.weights, caches[0].weights)
    # the graph goes by the lengths of its replay
    shorter = torch.tensor([700, 90, 30], dtype=torch.int32)
    caches[3].kv_lens.copy_(shorter)
    graphs[0].replay()
    again = sala_gla.paged_attention(d, caches[5].with_requests(caches[5].block_table, shorter.cuda()), SCALE, cu_seqlens=dcu)
    torch.cuda.synchronize()
    assert torch.equal(got[2][0], again[0]) and torch.equal(got[2][1], again[1])
    assert sala_gla.get_device_status() == 0


def test_bad_tables_lengths_and_offsets():
    from gated_linear_attention_gb300 import sala_gla
    q, cu = new_tokens([2, 20], 32, size=2.0)
    for bad in (-1, 5000, 2 ** 31 - 1, -2 ** 31):
        c = make_cache([90, 300], 16, 2, seed=4, weights=True)
        good = sala_gla.paged_attention(q.cuda(), on_gpu(c), SCALE, cu_seqlens=cu.cuda())
        c["table"][1, 7] = bad
        g = on_gpu(c)
        for accumulate in (False, True):
            o, _ = sala_gla.paged_attention(q.cuda(), g, SCALE, cu_seqlens=cu.cuda(), accumulate=accumulate)
            assert sala_gla.get_device_status() == 8
            assert torch.equal(o[:2], good[0][:2])
    c = make_cache([90, 300], 16, 2, seed=4)
    c["lens"][0] = 16 * c["table"].shape[1] + 1
    o, lse = sala_gla.paged_attention(q.cuda(), on_gpu(c), SCALE, cu_seqlens=cu.cuda())
    assert sala_gla.get_device_status() == 8
    assert bool((o[:2] == 0).all()) and bool((lse[:2] == -math.inf).all()) and torch.equal(o[2:], good[0][2:])
    c = make_cache([90, 300], 16, 2, seed=4)
    for bad in ([0, 3, 2], [0, -1, 22], [0, 2, 23], [5, 2, 22]):
        sala_gla.paged_attention(q.cuda(), on_gpu(c), SCALE, cu_seqlens=torch.tensor(bad, dtype=torch.int64).cuda())
        assert sala_gla.get_device_status() == 6


def test_nothing_to_do():
    from gated_linear_attention_gb300 import sala_gla
    c = on_gpu(make_cache([20, 20], 16, 2))
    o, lse = sala_gla.paged_attention(torch.zeros(2, 0, 32, 128, dtype=torch.bfloat16, device="cuda"), c, SCALE)
    assert tuple(o.shape) == (2, 0, 32, 128) and tuple(lse.shape) == (2, 0, 32)
    none = c.with_requests(c.block_table[:0], c.kv_lens[:0])
    o, _ = sala_gla.paged_attention(torch.zeros(0, 3, 32, 128, dtype=torch.bfloat16, device="cuda"), none, SCALE)
    assert o.numel() == 0


def test_refusals():
    from gated_linear_attention_gb300 import sala_gla
    raw = make_cache([20, 20], 16, 2)
    c = on_gpu(raw)
    q = torch.zeros(2, 1, 32, 128, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int64, device="cuda")
    for call, err in ((lambda: sala_gla.paged_attention(q.float(), c, SCALE), TypeError),
                      (lambda: sala_gla.paged_attention(q[:1], c, SCALE), ValueError),
                      (lambda: sala_gla.paged_attention(q[..., :31, :], c, SCALE), ValueError),
                      (lambda: sala_gla.paged_attention(q[:, 0], c, SCALE), ValueError),
                      (lambda: sala_gla.paged_attention(q[:, 0], c, SCALE, cu_seqlens=cu[:2]), ValueError),
                      (lambda: sala_gla.paged_attention(q[:, 0], c, SCALE, cu_seqlens=cu.int()), TypeError),
                      (lambda: sala_gla.paged_attention(q, c, SCALE, accumulate=True), ValueError),
                      (lambda: sala_gla.paged_attention(q, c, 0.0), sala_gla.SalaError),
                      (lambda: sala_gla.paged_attention(q, c, -1.0), sala_gla.SalaError),
                      (lambda: sala_gla.paged_attention(q, c, math.inf), sala_gla.SalaError),
                      (lambda: sala_gla.paged_attention(q, c, SCALE, o=q), sala_gla.SalaError),
                      (lambda: sala_gla.paged_attention(q.transpose(1, 2), c, SCALE), ValueError),
                      (lambda: on_gpu(dict(raw, k_pages=raw["k_pages"][:, :, :15])), ValueError),
                      (lambda: on_gpu(dict(raw, k_scale=torch.ones(2))), ValueError),
                      (lambda: on_gpu(dict(raw, table=raw["table"].long())), TypeError),
                      (lambda: on_gpu(dict(raw, lens=raw["lens"][:1])), ValueError)):
        with pytest.raises(err):
            call()
