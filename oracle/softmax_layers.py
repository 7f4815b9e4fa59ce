"""Plain forms, in 64 bits on the CPU, of the softmax layers' operators and of token scores: appending to a
paged cache, causal attention over it, eviction by accumulated weight, log probabilities. Written from the
definitions, request by request; shares no code with the library."""
import math

import torch

E4M3_MAX = 448.0


class Cache:
    """CPU copies of a paged cache; pages hold stored values (e4m3 ones as the 8-bit floats' values)."""

    def __init__(self, k_pages, v_pages, table, lens, k_scale=None, v_scale=None, weights=None):
        self.e4m3 = k_pages.dtype == torch.float8_e4m3fn
        self.k, self.v = (p.detach().cpu().to(torch.float32).double() for p in (k_pages, v_pages))
        self.table, self.lens = table.cpu().tolist(), lens.cpu().tolist()
        one = torch.ones(self.k.shape[1], dtype=torch.float64)
        self.k_scale, self.v_scale = (one if s is None else s.cpu().double() for s in (k_scale, v_scale))
        self.w = None if weights is None else weights.cpu().double()
        self.S = self.k.shape[2]

    def slot(self, n, i):
        return self.table[n][i // self.S], i % self.S

    def rows(self, pages, scale, n, h, end):
        out = [pages[p, h, s] * scale[h] for p, s in (self.slot(n, i) for i in range(end))]
        return torch.stack(out) if out else torch.zeros(0, pages.shape[-1], dtype=torch.float64)


def spans(cache, T, cu=None):
    """(first packed token, number of tokens) of each request."""
    if cu is None:
        return [(n * T, T) for n in range(len(cache.lens))]
    cu = cu.cpu().tolist()
    return [(a, b - a) for a, b in zip(cu, cu[1:])]


def append(cache, k, v, cu=None):
    T = k.shape[-3]
    k, v = (x.detach().cpu().reshape(-1, *x.shape[-2:]) for x in (k, v))
    for n, (first, count) in enumerate(spans(cache, T, cu)):
        for t in range(count):
            i = cache.lens[n] - count + t
            if i < 0:
                continue
            page, slot = cache.slot(n, i)
            for x, pages, scale in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
                y = x[first + t].float()
                if cache.e4m3:
                    y = (y / scale.float()[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float()
                pages[page, :, slot] = y.double()
            if cache.w is not None:
                cache.w[page, :, slot] = 0.0


def attend(cache, q, scale, cu=None, accumulate=False):
    """(o, lse, bounds): per element of o the sum of |p v|, per row the largest scale * sum |q k|. Tokens that
    no request has are NaN."""
    T, Hq = q.shape[-3], q.shape[-2]
    H = cache.k.shape[1]
    x = q.detach().cpu().double().reshape(-1, Hq, 128)
    o, mass = torch.full_like(x, math.nan), torch.zeros_like(x)
    lse, size = torch.full(x.shape[:2], math.nan, dtype=torch.float64), torch.zeros(x.shape[:2], dtype=torch.float64)
    for n, (first, count) in enumerate(spans(cache, T, cu)):
        end = cache.lens[n]
        for h in range(H if count else 0):
            ks, vs = cache.rows(cache.k, cache.k_scale, n, h, end), cache.rows(cache.v, cache.v_scale, n, h, end)
            heads = slice(h * (Hq // H), (h + 1) * (Hq // H))
            slots = torch.tensor([cache.slot(n, i) for i in range(end)], dtype=torch.long).reshape(-1, 2)
            for t in range(count):
                seen, row = max(0, end - count + t + 1), x[first + t, heads]
                if not seen:
                    o[first + t, heads], lse[first + t, heads] = 0.0, -math.inf
                    continue
                s = scale * (row @ ks[:seen].T)
                lse[first + t, heads] = s.logsumexp(1)
                p = (s - lse[first + t, heads, None]).exp()
                o[first + t, heads] = p @ vs[:seen]
                mass[first + t, heads] = p @ vs[:seen].abs()
                size[first + t, heads] = scale * (row.abs() @ ks[:seen].abs().T).amax(1)
                if accumulate:
                    cache.w[slots[:seen, 0], h, slots[:seen, 1]] += p.sum(0)
    return o.reshape(q.shape), lse.reshape(q.shape[:-1]), (mass.reshape(q.shape), size.reshape(q.shape[:-1]))


def evict(cache, budget, sinks, recent):
    """(new lengths, kept [N, H, budget])."""
    N, H = len(cache.lens), cache.k.shape[1]
    kept = torch.full((N, H, budget), -1, dtype=torch.int32)
    for n, end in enumerate(cache.lens):
        for h in range(H):
            if end <= budget:
                kept[n, h, :end] = torch.arange(end, dtype=torch.int32)
                continue
            def weight(i):
                w = float(cache.w[cache.slot(n, i)[0], h, cache.slot(n, i)[1]])
                return w if w > 0 else 0.0
            middle = sorted(range(sinks, end - recent), key=lambda i: (-weight(i), i))[:budget - sinks - recent]
            stay = list(range(sinks)) + sorted(middle) + list(range(end - recent, end))
            kept[n, h] = torch.tensor(stay, dtype=torch.int32)
            src = [cache.slot(n, i) for i in stay]
            for pages in (cache.k, cache.v, cache.w):
                moved = [pages[p, h, s].clone() for p, s in src]
                for i, x in enumerate(moved):
                    page, slot = cache.slot(n, i)
                    pages[page, h, slot] = x
    return torch.tensor([min(x, budget) for x in cache.lens], dtype=torch.int32), kept


def logprobs(logits, tokens, top=0):
    """(logprobs, entropy, top tokens, top logprobs); NaN counts as -inf, +inf as the largest float."""
    x = logits.detach().cpu().double()
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x).clamp(max=torch.finfo(torch.float32).max)
    d = x - x.amax(1, keepdim=True)      # first: log sum exp itself would be lost beside the largest floats
    lp = d - d.logsumexp(1, keepdim=True)
    lp = torch.where(lp.isnan(), torch.full_like(lp, -math.inf), lp)
    entropy = -torch.where(lp > -math.inf, lp.exp() * lp, torch.zeros_like(lp)).sum(1)
    out = None
    if tokens is not None:
        t = tokens.cpu().long().reshape(x.shape[0], -1)
        ok = (t >= 0) & (t < x.shape[1])
        out = torch.where(ok, lp.gather(1, t.clamp(0, x.shape[1] - 1)), torch.zeros(t.shape, dtype=torch.float64))
        out = out.reshape(tokens.shape)
    ids = torch.full((x.shape[0], top), -1, dtype=torch.int32)
    values = torch.full((x.shape[0], top), -math.inf, dtype=torch.float64)
    for n in range(x.shape[0]):
        order = sorted((i for i in range(x.shape[1]) if x[n, i] > -math.inf), key=lambda i: (-float(x[n, i]), i))[:top]
        for r, i in enumerate(order):
            ids[n, r], values[n, r] = i, lp[n, i]
    return out, entropy, ids, values
