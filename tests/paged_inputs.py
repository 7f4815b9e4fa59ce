"""Seeded paged caches for the tests of the softmax layers' operators."""
import torch

D = 128


def make_cache(lens, page=16, H=2, kind="bf16", seed=0, spare=2, weights=False, width=None, stale=None, past=-1):
    """CPU tensors of a cache whose requests have `lens` tokens: pages in random order, table entries
    past a length `past`, unused rows of pages (and pages nobody has) `stale` where that is given."""
    gen = torch.Generator().manual_seed(seed)
    N, need = len(lens), [-(-x // page) for x in lens]
    width = max(1, max(need, default=1)) if width is None else width
    P = sum(need) + spare
    order = torch.randperm(P, generator=gen).tolist()
    table = torch.full((N, width), past, dtype=torch.int32)
    k, v = torch.randn(P, H, page, D, generator=gen), torch.randn(P, H, page, D, generator=gen)
    used = torch.zeros(P, page, dtype=torch.bool)
    for n, count in enumerate(need):
        for i in range(count):
            p = order.pop()
            table[n, i] = p
            used[p, :min(page, lens[n] - i * page)] = True
    out = dict(table=table, lens=torch.tensor(lens, dtype=torch.int32), k_scale=None, v_scale=None)
    if kind == "e4m3":
        out["k_scale"], out["v_scale"] = (0.01 + 0.02 * torch.rand(H, generator=gen) for _ in range(2))
        # a cast alone makes NaN of what is above 448
        k, v = ((x / s[:, None, None]).clamp(-448, 448) for x, s in ((k, out["k_scale"]), (v, out["v_scale"])))
    if stale is not None:
        for x in (k, v):
            x.masked_fill_(~used[:, None, :, None], stale)
    dt = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    out["k_pages"], out["v_pages"] = k.to(dt), v.to(dt)
    out["weights"] = torch.rand(P, H, page, generator=gen) if weights else None
    return out


def on_gpu(c):
    from gated_linear_attention_gb300 import sala_gla
    d = {n: None if t is None else t.cuda() for n, t in c.items()}
    return sala_gla.KvCache(d["k_pages"], d["v_pages"], d["table"], d["lens"], d["k_scale"], d["v_scale"], d["weights"])


def on_cpu(c):
    from oracle import softmax_layers as ref
    return ref.Cache(c["k_pages"], c["v_pages"], c["table"], c["lens"], c["k_scale"], c["v_scale"], c["weights"])


def new_tokens(counts, heads, seed=1, size=1.0):
    """Packed bf16 [T, heads, 128] and int64 offsets."""
    gen = torch.Generator().manual_seed(seed)
    cu = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0)
    return (size * torch.randn(int(cu[-1]), heads, D, generator=gen)).to(torch.bfloat16), cu


def bits(t):
    """Integers of a tensor's bits, for comparisons that NaN does not escape."""
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()
