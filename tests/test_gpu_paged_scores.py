"""Attention over a paged cache at every scale that is allowed, from weights that are all alike to a largest score that is
all that counts, with e4m3 keys of large and small scales.

Queries and keys are small whole numbers (times a power of two for e4m3), so that the scores s = q.k are exact in fp32 and ties are
ties. What remains, with c = scale * k_scale * log2 e (relative error d <= 4 * 2^-24, from its roundings) and m the largest score:
  - exponents c (s - m): those below -150 give 0, the others are off by 150 (d + 2^-24) at most; where |c m| <= 1024 the rounding of
    c m is common to all of a row but for maxima that grew, by 2^8 at least, and so leaves 2 * 1024 * 2^-24 * 2^-8. Times log 2: 2^-15.
  - exp2 2^-21; sums of n positive terms in chains of at most 128 + n / 128: E = 2^-15 + 2^-21 + (128 + n / 128) 2^-24 of a weight's
    numerator or of their sum. o: as in test_gpu_paged_attention.py, with this E.
  - lse = (c m + log2 sum) log 2: E and its roundings (c's, the product, the sum, log 2, the product) 6 * 2^-24 |lse|.
  - accumulated weights go by z = m + log2(sum) / c, rounded: a relative error of |lse| 2^-23 beside 2 E. Where that is large the
    rounding still leaves m <= z <= m + 2 log2(sum) / c: a weight lies between p / sum and p * sum."""
import math

import pytest
import torch

from paged_inputs import make_cache, new_tokens, on_cpu, on_gpu

pytestmark = pytest.mark.gpu
SCALES = [1e-18, 1e-6, 0.088, 1.0, 37.0, 1e3, 1e5, 1e7, 1e9, 1e12, 1e18]


def _whole_numbers(lens, T, Hq, H, kind, k_scale, seed):
    c = make_cache(lens, 16, H, kind, seed=seed, weights=True)
    gen = torch.Generator().manual_seed(seed)
    c["k_pages"] = torch.randint(-3, 4, c["k_pages"].shape, generator=gen).float().to(c["k_pages"].dtype)
    c["weights"].zero_()
    if kind == "e4m3":
        c["k_scale"] = torch.tensor([k_scale, 1.0] * H)[:H]
    q = torch.randint(-3, 4, (len(lens), T, Hq, 128), generator=gen).to(torch.bfloat16)
    return c, q


def _exact(r, q, scale):
    """o, lse, sum |p v|, and as r.w is laid out the sums over the rows of p, of p / sum and of p * sum. The largest score is taken off
    before the scale: beside log sum exp itself (1e33 here) 64 bits lose the rest."""
    N, T, Hq, _ = q.shape
    H = r.k.shape[1]
    G = Hq // H
    o, mass, lse = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64), torch.zeros(N, T, Hq, dtype=torch.float64)
    sums, low, high = (torch.zeros_like(r.k[..., 0]) for _ in range(3))
    for n in range(N):
        end = r.lens[n]
        for h in range(H):
            ks, vs = r.rows(r.k, torch.ones(H, dtype=torch.float64), n, h, end), r.rows(r.v, r.v_scale, n, h, end)
            slots = torch.tensor([r.slot(n, i) for i in range(end)])
            for t in range(T):
                seen, heads = end - T + t + 1, slice(h * G, (h + 1) * G)
                s = q[n, t, heads].double() @ ks[:seen].T
                top, unit = s.amax(1, keepdim=True), scale * float(r.k_scale[h])
                e = (unit * (s - top)).exp()
                total = e.sum(1, keepdim=True)
                lse[n, t, heads] = (unit * top + total.log())[:, 0]
                o[n, t, heads], mass[n, t, heads] = e / total @ vs[:seen], e / total @ vs[:seen].abs()
                for out, x in ((sums, e / total), (low, e / total ** 2), (high, e)):
                    out[slots[:seen, 0], h, slots[:seen, 1]] += x.sum(0)
    return o, lse, mass, sums, low, high


@pytest.mark.parametrize("kind,k_scale", [("bf16", 1.0), ("e4m3", 1.0), ("e4m3", 2.0 ** 39), ("e4m3", 2.0 ** -39)])
@pytest.mark.parametrize("T,Hq,H,lens", [(1, 8, 2, [3000, 17]), (5, 8, 1, [700]), (40, 16, 2, [300, 41]), (1, 4, 1, [9, 300, 130] * 60)])
def test_scales(kind, k_scale, T, Hq, H, lens):
    from gated_linear_attention_gb300 import sala_gla
    for scale in SCALES:
        c, q = _whole_numbers(lens, T, Hq, H, kind, k_scale, seed=T)
        g, r = on_gpu(c), on_cpu(c)
        o, lse = sala_gla.paged_attention(q.cuda(), g, scale, accumulate=True)
        assert sala_gla.get_device_status() == 0
        exact = float(torch.tensor(scale, dtype=torch.float32))
        ro, rlse, mass, sums, low, high = _exact(r, q, exact)
        E = 2.0 ** -15 + 2.0 ** -21 + (128 + max(lens) / 128) * 2.0 ** -24
        err = (o.cpu().double() - ro).abs()
        assert bool((err <= (2.0 ** -8 + 2 * E + 2.0 ** -16) * mass + 2.0 ** -8 * ro.abs()).all()), (scale, float(err.max()))
        err = (lse.cpu().double() - rlse).abs()
        assert bool((err <= E + 6 * 2.0 ** -24 * rlse.abs()).all()), (scale, float(err.max()))
        w, rows = g.weights.cpu().double(), T * Hq // H
        e = 2 * E + 2.0 ** -21 + rows * 2.0 ** -23
        assert bool((w >= low * (1 - e) - 1e-30).all()) and bool((w <= high * (1 + e) + 1e-30).all()), scale
        off = float(rlse.abs().max()) * 2.0 ** -23
        if off < 0.1:
            assert bool(((w - sums).abs() <= (e + 2 * off) * sums + 1e-30).all()), (scale, float((w - sums).abs().max()))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,L", [(1, 2500), (7, 700), (40, 300)])
@pytest.mark.parametrize("scale", [1e6, 1e9, 1e18])
def test_largest_score_is_all_that_counts(kind, T, L, scale):
    """Scores with roundings, at most 128 * 2^-24 sum |q k|: rows whose largest score leads by more give that place's values,
    and no weight passes the number of rows."""
    from gated_linear_attention_gb300 import sala_gla
    c = make_cache([L], 32, 1, kind, seed=T, weights=True)
    c["weights"].zero_()
    q, _ = new_tokens([T], 8, seed=2, size=2.0)
    g, r = on_gpu(c), on_cpu(c)
    o, lse = sala_gla.paged_attention(q[None].cuda(), g, scale, accumulate=True)
    assert sala_gla.get_device_status() == 0
    ks, vs = r.rows(r.k, r.k_scale, 0, 0, L), r.rows(r.v, r.v_scale, 0, 0, L)
    checked = 0
    for t in range(T):
        seen = L - T + t + 1
        s = q[t].double() @ ks[:seen].T
        bound = 2 * 128 * 2.0 ** -24 * (q[t].double().abs() @ ks[:seen].abs().T).amax(1) + 150 / scale
        top, at = s.topk(2, dim=1)
        for h in range(8):
            if float(top[h, 0] - top[h, 1]) > float(bound[h]):
                checked += 1
                want = vs[at[h, 0]]
                assert bool(((o[0, t, h].cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-30).all())
                assert abs(float(lse[0, t, h]) - scale * float(top[h, 0])) <= scale * float(bound[h]) + 6 * 2.0 ** -24 * scale * float(top[h, 0])
    assert checked > 4
    assert bool(o.isfinite().all()) and bool(lse.isfinite().all())
    assert float(g.weights.max()) <= 8 * T and float(g.weights.min()) >= 0 and float(g.weights.sum()) >= checked
