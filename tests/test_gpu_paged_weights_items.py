"""Accumulated weights of many short prompts: blocks that go through dozens of cache tiles with one to eight query tiles each, whose
partial sums the groups hand to one another. Against the plain form in 64 bits (here over padded requests), and the
same bits every time. Bounds as in test_gpu_paged_attention.py."""
import random

import pytest
import torch

from paged_inputs import make_cache, on_gpu

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def _plain(c, q, counts):
    """(sums of weights of the places [N, H, L], the largest error E of a score or sum)."""
    N, H, S = len(counts), c["k_pages"].shape[1], c["k_pages"].shape[2]
    G, L, most = q.shape[1] // H, int(c["lens"].max()), max(counts)
    k = c["k_pages"].cuda().float().double()
    if c["k_scale"] is not None:
        k = k * c["k_scale"].cuda().double()[:, None, None]
    at = torch.arange(L)
    page = c["table"][:, at // S].clamp(min=0).long()                       # [N, L]
    k = k[page.cuda(), :, (at % S).cuda()].permute(0, 2, 1, 3)             # [N, H, L, 128]
    rows = torch.zeros(N, most, q.shape[1], 128, dtype=torch.float64, device="cuda")
    first = 0
    for n, count in enumerate(counts):
        rows[n, :count] = q[first:first + count].double()
        first += count
    x = rows.view(N, most, H, G, 128).permute(0, 2, 1, 3, 4).reshape(N, H, most * G, 128)
    s = SCALE * x @ k.transpose(2, 3)
    size = float((SCALE * x.abs() @ k.abs().transpose(2, 3)).max())
    lens, count = c["lens"].cuda().long(), torch.tensor(counts, device="cuda")
    t = torch.arange(most, device="cuda")
    limit = torch.where(t < count[:, None], lens[:, None] - count[:, None] + t, -1).repeat_interleave(G, 1)   # [N, rows]
    p = s.masked_fill(at.cuda() > limit[:, None, :, None], -torch.inf).softmax(-1).nan_to_num(0.0)
    return p.sum(2), 128 * 2.0 ** -24 * size + 2.0 ** -21 + (128 + L / 128) * 2.0 ** -24


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("N,Hq,H,most", [(500, 128, 8, 60), (200, 128, 8, 60), (256, 64, 4, 33), (61, 128, 1, 20)])
def test_many_items(kind, N, Hq, H, most):
    from gated_linear_attention_gb300 import sala_gla
    rng = random.Random(N + most)
    lens = [rng.randint(0, 40) if rng.random() < 0.8 else rng.randint(100, 300) for _ in range(N)]
    counts = [rng.choice((0, 1, 5, rng.randint(0, most), rng.randint(0, min(x, most)))) for x in lens]
    counts[3] = most
    c = make_cache(lens, 64, H, kind, seed=N, weights=True)
    gen = torch.Generator(device="cuda").manual_seed(N)
    q = (2 * torch.randn(sum(counts), Hq, 128, generator=gen, device="cuda")).to(torch.bfloat16)
    cu = torch.tensor([0] + counts, device="cuda").cumsum(0)
    sums, E = _plain(c, q, counts)
    was, want = c["weights"].double(), c["weights"].double()
    for n in range(N):
        i = torch.arange(lens[n])
        want[c["table"][n, i // 64].long(), :, i % 64] += sums[n, :, :lens[n]].T.cpu()
    first = None
    for _ in range(8):
        g = on_gpu(c)
        sala_gla.paged_attention(q, g, SCALE, cu_seqlens=cu, accumulate=True)
        assert sala_gla.get_device_status() == 0
        got = g.weights.cpu()
        first = got if first is None else first
        assert torch.equal(got, first)
        err = (got.double() - want).abs()
        bound = (2 * E + 2.0 ** -21 + most * Hq // H * 2.0 ** -24) * (want - was) + 2.0 ** -24 * want
        assert bool((err <= bound).all()), float(err.max())
