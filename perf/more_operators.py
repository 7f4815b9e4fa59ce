"""Workloads of the softmax layers between the Simple GLA layers, and of scoring what a model answers.

Four operators, each in a plain form (elementary torch operations) and as the library's call:

append    keys and values of new tokens into the pages of a paged cache, bf16 or e4m3 with a scale a head
attend    attention of a chunk of new tokens over the cache (one token each while decoding, drafted tokens,
          chunks of prompts), on request with each cached token's attention weight added to its running sum
evict     eviction by that sum: the heaviest tokens, the first and the newest stay, moved together in order
logprobs  log probabilities of given tokens, the entropy and the top alternatives of each row of logits

Shapes are those of the softmax layers next to the lightning layers (32 query heads on 2 key/value heads of
dimension 128) and other head layouts around them, pages of 16 to 256 tokens.
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


def listed():
    return [
        # one user, one new token: latency
        dict(name="append_one", op="append", N=1, T=1, L=4001, Hkv=2, page=16, type="bf16", ragged=False),
        # prompts of different lengths into an e4m3 cache
        dict(name="append_prompts", op="append", N=13, T=4999, L=8192, Hkv=2, page=64, type="e4m3", ragged=True),
        # one user, decoding
        dict(name="attend_one", op="attend", N=1, T=1, L=4001, Hq=32, Hkv=2, page=16, type="bf16", ragged=False,
             accumulate=False),
        # a full serving batch, decoding at different lengths
        dict(name="attend_batch", op="attend", N=256, T=1, L=12288, Hq=32, Hkv=2, page=64, type="bf16", ragged=True,
             accumulate=False),
        # five drafted tokens a request on an e4m3 cache that evicts by weight
        dict(name="attend_drafts", op="attend", N=61, T=5, L=8192, Hq=32, Hkv=2, page=128, type="e4m3", ragged=False,
             accumulate=True),
        # a chunk of a long prompt
        dict(name="attend_chunk", op="attend", N=1, T=4096, L=32768, Hq=32, Hkv=2, page=64, type="bf16", ragged=False,
             accumulate=False),
        # chunks of several prompts at different places, weights summed for a later eviction
        dict(name="attend_prompts", op="attend", N=7, T=2011, L=6007, Hq=32, Hkv=2, page=16, type="bf16", ragged=True,
             accumulate=True),
        # a few requests back to a budget
        dict(name="evict_few", op="evict", N=3, L=700, budget=512, sinks=4, recent=64, Hkv=2, page=16, type="bf16"),
        # a batch cut to half of its cache
        dict(name="evict_batch", op="evict", N=96, L=8192, budget=4096, sinks=16, recent=1024, Hkv=2, page=64,
             type="bf16"),
        # one row, with its alternatives: latency
        dict(name="logprobs_one", op="logprobs", N=1, V=65536, M=1, top=5, type="f32"),
        # every token of a prompt scored; odd vocabulary, rows off 16-byte boundaries
        dict(name="logprobs_prompt", op="logprobs", N=2048, V=50021, M=1, top=0, type="bf16"),
        # a full batch with alternatives
        dict(name="logprobs_batch", op="logprobs", N=256, V=131072, M=3, top=20, type="f32"),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "attend", "attend", "evict", "evict", "logprobs", "logprobs"))
    if op == "logprobs":
        N, V = _between(rng, 1, 2048), _between(rng, 2000, 131072)
        N = max(1, min(N, 256 * 131072 // V))
        return dict(op=op, N=N, V=V, M=rng.randint(1, 5), top=rng.choice((0, 1, 5, 10, 20, 32)),
                    type=rng.choice(("f32", "bf16")))
    kind, page = rng.choice(("bf16", "e4m3")), rng.choice((16, 32, 64, 128, 256))
    Hq, Hkv = rng.choice(((32, 2), (32, 2), (8, 8), (16, 4), (24, 2), (40, 8), (5, 1), (14, 2), (64, 1)))
    if op == "append":
        L = _between(rng, 40, 8192)
        return dict(op=op, N=_between(rng, 1, 16), T=_between(rng, 1, L), L=L, Hkv=Hkv, page=page, type=kind,
                    ragged=rng.random() < 0.6)
    if op == "evict":
        L = _between(rng, 80, 8192)
        budget = max(16, int(L * rng.uniform(0.2, 0.95)))
        sinks = rng.choice((0, 1, 4, 16))
        return dict(op=op, N=_between(rng, 1, 96), L=L, budget=budget, sinks=sinks,
                    recent=rng.randint(0, (budget - sinks) // 2), Hkv=min(Hkv, 4), page=page, type=kind)
    L = _between(rng, 50, 32768)
    T = 1 if rng.random() < 0.3 else rng.randint(2, min(L, 17)) if rng.random() < 0.4 else _between(rng, 2, min(L, 4096))
    most = min(256, 8e9 / (Hq * T * L * 4), 256 * 8192 * 2 / (L * Hkv))
    return dict(op=op, N=_between(rng, 1, max(1, int(most))), T=T, L=L, Hq=Hq, Hkv=Hkv, page=page, type=kind,
                ragged=rng.random() < 0.6, accumulate=rng.random() < 0.4)


# ---- inputs --------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "logprobs":
        return _prepare_logprobs(case, gen)
    return _prepare_cache(case, gen)


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda")


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _ints(gen, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int32)


def _lengths(c, gen):
    """Tokens in the cache (the new ones among them) and new tokens of each request."""
    N, L, T = c["N"], c["L"], c.get("T", 1)
    if c["op"] == "evict":
        lens = _ints(gen, max(1, min(c["budget"], 3 * L // 4)), L + 1, N)
        lens[0] = L
        return lens, torch.zeros_like(lens)
    if not c["ragged"]:
        return torch.full((N,), L, dtype=torch.int32, device="cuda"), torch.full((N,), T, dtype=torch.int32, device="cuda")
    # the numbers of new tokens are the case's own: outputs have the same shape for every seed
    new = _ints(torch.Generator(device="cuda").manual_seed(N * 8191 + T), max(1, T // 4), T + 1, N)
    lens = torch.maximum(_ints(gen, max(1, L // 3), L + 1, N), new)
    lens[N - 1], new[0] = L, T
    lens[0] = torch.maximum(lens[0], new[0])
    if N > 2:
        new[N // 2] = 0    # a request of the batch with nothing new
    return lens, new


def _prepare_cache(c, gen):
    N, L, Hkv, S, kind = c["N"], c["L"], c["Hkv"], c["page"], TYPES[c["type"]]
    lens, new = _lengths(c, gen)
    width = -(-L // S)
    P = N * width + 3
    table = torch.randperm(P, generator=gen, device="cuda")[:N * width].to(torch.int32).reshape(N, width)
    s = dict(op=c["op"], table=table, lens=lens)
    k, v = _randn(gen, P, Hkv, S, D), _randn(gen, P, Hkv, S, D)
    if c["type"] == "e4m3":
        s["k_scale"], s["v_scale"] = 0.01 + 0.02 * _rand(gen, Hkv), 0.01 + 0.02 * _rand(gen, Hkv)
        k, v = (_quantised(t, sc[:, None, None], kind) for t, sc in ((k, s["k_scale"]), (v, s["v_scale"])))
    else:
        s["k_scale"] = s["v_scale"] = None
        k, v = k.to(kind), v.to(kind)
    s["k_pages"], s["v_pages"], s["weights"] = k, v, None
    if c["op"] == "evict":
        # running sums with a long tail, and tokens that never had any
        w = (1.5 * _randn(gen, P, Hkv, S)).exp()
        s["weights"] = torch.where(_rand(gen, P, Hkv, S) < 0.2, torch.zeros_like(w), w)
        return dict(s, budget=c["budget"], sinks=c["sinks"], recent=c["recent"])
    cu = torch.zeros(N + 1, dtype=torch.int64, device="cuda")
    cu[1:] = new.cumsum(0)
    # equal numbers of new tokens come as [N, T, ...], others packed with cu_seqlens
    lead = (int(cu[-1]),) if c["ragged"] else (N, c["T"])
    s["cu"], s["T"] = cu if c["ragged"] else None, c["T"]    # T: the most new tokens of a request
    if c["op"] == "append":
        return dict(s, k=_randn(gen, *lead, Hkv, D).to(torch.bfloat16), v=_randn(gen, *lead, Hkv, D).to(torch.bfloat16))
    if c["accumulate"]:
        s["weights"] = _rand(gen, P, Hkv, S)
    return dict(s, q=(2.5 * _randn(gen, *lead, c["Hq"], D)).to(torch.bfloat16), accumulate=c["accumulate"])


def _quantised(x, scale, kind):
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(kind)


def _prepare_logprobs(c, gen):
    """Peaked logits, and tokens that were drawn from them."""
    x = (3.0 * _randn(gen, c["N"], c["V"])).to(TYPES[c["type"]])
    tokens = torch.multinomial(x.float().softmax(-1), c["M"], generator=gen).to(torch.int32)
    return dict(op="logprobs", x=x, tokens=tokens, top=c["top"])


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"append": _plain_append, "attend": _plain_attend, "evict": _plain_evict,
            "logprobs": _plain_logprobs}[state["op"]](state)


def _run_own(s):
    from gated_linear_attention_gb300 import sala_gla
    if s["op"] == "logprobs":
        got = sala_gla.token_logprobs(s["x"], s["tokens"], top=s["top"])
        return dict(zip(("logprobs", "entropy", "top_tokens", "top_logprobs"), got))
    cache = sala_gla.KvCache(s["k_pages"], s["v_pages"], s["table"], s["lens"], k_scale=s["k_scale"],
                             v_scale=s["v_scale"], weights=s["weights"])
    if s["op"] == "append":
        sala_gla.kv_append(cache, s["k"], s["v"], cu_seqlens=s["cu"])
        return dict(k=s["k_pages"], v=s["v_pages"])
    if s["op"] == "attend":
        o, lse = sala_gla.paged_attention(s["q"], cache, SCALE, cu_seqlens=s["cu"], accumulate=s["accumulate"])
        return dict(o=o, lse=lse, weights=s["weights"] if s["accumulate"] else None)
    lens, kept = sala_gla.kv_evict(cache, s["budget"], sinks=s["sinks"], recent=s["recent"])
    return dict(lens=lens, kept=kept, k=s["k_pages"], v=s["v_pages"], weights=s["weights"])


def _new_places(s):
    """For each packed new token: its request and its place in the cache."""
    if s["cu"] is None:
        N, T = s["lens"].numel(), s["T"]
        first = torch.arange(N, device="cuda") * T
        counts = torch.full((N,), T, device="cuda")
        total = N * T
    else:
        first, counts = s["cu"][:-1], s["cu"].diff()
        total = s["q" if "q" in s else "k"].shape[0]
    t = torch.arange(total, device="cuda")
    seq = torch.searchsorted(first + counts, t, right=True)
    return seq, t - first[seq] + s["lens"].long()[seq] - counts[seq]


def _plain_append(s):
    seq, place = _new_places(s)
    S = s["k_pages"].shape[2]
    page = s["table"].long()[seq, place // S]
    for name in ("k", "v"):
        x, pages, scale = s[name].reshape(-1, *s[name].shape[-2:]), s[name + "_pages"], s[name + "_scale"]
        if scale is None:
            pages[page, :, place % S] = x
        else:   # bytes are stored: indexing is not defined for 8-bit floats everywhere
            stored = _quantised(x.float(), scale[:, None], pages.dtype)
            pages.view(torch.uint8)[page, :, place % S] = stored.view(torch.uint8)
    return dict(k=s["k_pages"], v=s["v_pages"])


def _gathered(pages, table, scale):
    """[N, Hkv, places, 128] in 32 bits."""
    x = pages.view(torch.uint8)[table.long()].view(torch.float8_e4m3fn) if scale is not None else pages[table.long()]
    N, W, H, S, _ = x.shape
    x = x.permute(0, 2, 1, 3, 4).reshape(N, H, W * S, -1).float()
    return x if scale is None else x * scale[:, None, None]


def _plain_attend(s):
    q, table, lens = s["q"], s["table"], s["lens"].long()
    Hq, (N, W) = q.shape[-2], table.shape
    k, v = _gathered(s["k_pages"], table, s["k_scale"]), _gathered(s["v_pages"], table, s["v_scale"])
    Hkv, L = k.shape[1], k.shape[2]
    G = Hq // Hkv
    seq, place = _new_places(s)
    most = s["T"]
    row = place - (lens[seq] - (most if s["cu"] is None else s["cu"].diff()[seq]))
    padded = torch.zeros(N, most, Hq, D, device="cuda")
    padded[seq, row] = q.reshape(-1, Hq, D).float()
    limit = torch.full((N, most), -1, dtype=torch.int64, device="cuda")   # the last place that a row sees
    limit[seq, row] = place
    at = torch.arange(L, device="cuda")
    hidden = at > limit[:, :, None]                                        # [N, T, L]
    rows = padded.reshape(N, most, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(N, Hkv, most * G, D)
    x = torch.matmul(rows, k.transpose(2, 3)).mul_(SCALE).reshape(N, Hkv, most, G, L)
    x.masked_fill_(hidden[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0].permute(0, 2, 1, 3).reshape(N, most, Hq)
    x /= total.clamp(min=1e-30)
    o = torch.matmul(x.reshape(N, Hkv, most * G, L), v).reshape(N, Hkv, most, G, D).permute(0, 2, 1, 3, 4)
    o = o.reshape(N, most, Hq, D)[seq, row].to(torch.bfloat16).reshape(q.shape)
    lse = lse[seq, row].reshape(q.shape[:-1])
    if not s["accumulate"]:
        return dict(o=o, lse=lse, weights=None)
    S, w = s["k_pages"].shape[2], x.sum((2, 3))                            # [N, Hkv, L]
    live = (at < lens[:, None])[:, None].expand(N, Hkv, L)
    place = (table.long()[:, None, at // S] * Hkv + torch.arange(Hkv, device="cuda")[:, None]) * S + at % S
    s["weights"].view(-1)[place[live]] += w[live]
    return dict(o=o, lse=lse, weights=s["weights"])


def _plain_evict(s):
    table, lens, budget = s["table"], s["lens"].long(), s["budget"]
    S, Hkv = s["k_pages"].shape[2], s["k_pages"].shape[1]
    N, W = table.shape
    at = torch.arange(W * S, device="cuda")
    heads = torch.arange(Hkv, device="cuda")[:, None]
    place = (table.long()[:, None, at // S] * Hkv + heads) * S + at % S     # [N, Hkv, L]
    w = s["weights"].view(-1)[place]
    end = lens[:, None, None]
    w = torch.where((at < s["sinks"]) | (at >= end - s["recent"]), torch.full_like(w, math.inf), w)
    w = torch.where(at >= end, torch.full_like(w, -1.0), w)
    budget = min(budget, W * S)
    order = torch.sort(w, dim=2, descending=True, stable=True).indices[..., :budget]
    order = torch.where(order < end, order, torch.full_like(order, W * S))  # past the end: last
    kept = order.sort(2).values
    stays = kept < W * S
    src, dst = place.gather(2, kept.clamp(max=W * S - 1))[stays], place[..., :budget][stays]
    for name in ("k_pages", "v_pages"):
        flat = s[name].view(-1, D)
        flat = flat if s["k_scale"] is None else flat.view(torch.uint8)
        flat[dst] = flat[src]
    s["weights"].view(-1)[dst] = s["weights"].view(-1)[src]
    kept = torch.where(stays, kept, torch.full_like(kept, -1)).to(torch.int32)
    if budget < s["budget"]:
        kept = torch.nn.functional.pad(kept, (0, s["budget"] - budget), value=-1)
    return dict(lens=s["lens"].clamp(max=s["budget"]), kept=kept, k=s["k_pages"], v=s["v_pages"], weights=s["weights"])


def _plain_logprobs(s):
    x, top = s["x"].float(), s["top"]
    peak = x.amax(1, keepdim=True)
    e = (x - peak).exp()
    total = e.sum(1, keepdim=True)
    lse = peak + total.log()
    logprobs = x.gather(1, s["tokens"].long()) - lse
    entropy = (e * (lse - x)).sum(1) / total[:, 0]
    if not top:
        return dict(logprobs=logprobs, entropy=entropy, top_tokens=None, top_logprobs=None)
    values, ids = torch.sort(x, dim=1, descending=True, stable=True)       # ties: the lowest index
    return dict(logprobs=logprobs, entropy=entropy, top_tokens=ids[:, :top].to(torch.int32),
                top_logprobs=values[:, :top] - lse)


# ---- the definition in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "evict": _exact_evict,
            "logprobs": _exact_logprobs}[case["op"]](s)


def _values(pages, scale):
    x = pages.to(torch.float64)
    return x if scale is None else x * scale.double()[:, None, None]


def _counts(s):
    N = s["lens"].numel()
    return s["cu"].diff().tolist() if s["cu"] is not None else [s["T"]] * N


def _exact_append(s):
    """Values that are stored, unrounded, in units of the scale; page by page."""
    out, S = {}, s["k_pages"].shape[2]
    for name in ("k", "v"):
        pages, scale = s[name + "_pages"].to(torch.float64), s[name + "_scale"]
        x = s[name].reshape(-1, *s[name].shape[-2:]).double()
        if scale is not None:
            x = (x / scale.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        t = 0
        for n, (count, end) in enumerate(zip(_counts(s), s["lens"].tolist())):
            i = end - count
            while i < end:
                stop = min(end, (i // S + 1) * S)
                part = x[t:t + stop - i].transpose(0, 1)
                pages[int(s["table"][n, i // S]), :, i % S:i % S + stop - i] = part
                t, i = t + stop - i, stop
        out[name] = pages
    return out


def _exact_attend(s):
    """One request and one query head at a time, as the formula stands."""
    q = s["q"].reshape(-1, *s["q"].shape[-2:])
    Hq, Hkv, S = q.shape[1], s["k_pages"].shape[1], s["k_pages"].shape[2]
    G, t = Hq // Hkv, 0
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if s["accumulate"] else None
    for n, (count, end) in enumerate(zip(_counts(s), s["lens"].tolist())):
        used = s["table"][n, :-(-end // S)].tolist()
        past = torch.arange(end, device="cuda") > torch.arange(end - count, end, device="cuda")[:, None]
        for h in range(Hkv):
            k, v = (torch.cat([(p[page, h].to(torch.float32).double() * (1.0 if sc is None else sc[h].double()))
                               for page in used])[:end]
                    for p, sc in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])))
            sums = torch.zeros(end, dtype=torch.float64, device="cuda")
            for g in range(h * G, (h + 1) * G):
                x = (q[t:t + count, g].double() @ k.T / math.sqrt(D)).masked_fill_(past, -math.inf)
                lse[t:t + count, g] = x.logsumexp(1)
                x = x.sub_(lse[t:t + count, g, None]).exp_()
                o[t:t + count, g] = x @ v
                sums += x.sum(0)
            if weights is not None:
                for i, page in enumerate(used):
                    part = sums[i * S:(i + 1) * S]
                    weights[page, h, :part.numel()] += part
        t += count
    return dict(o=o.reshape(s["q"].shape), lse=lse.reshape(s["q"].shape[:-1]), weights=weights)


def _exact_evict(s):
    """Token by token for one request and head after another (values move, none is computed)."""
    S = s["k_pages"].shape[2]
    k, v, w = s["k_pages"].to(torch.float64), s["v_pages"].to(torch.float64), s["weights"].double()
    for n, end in enumerate(s["lens"].tolist()):
        places = torch.arange(end, device="cuda")
        page, slot = s["table"][n].long()[places // S], places % S
        count = min(end, s["budget"])
        for h in range(k.shape[1]):
            forced = [i for i in range(end) if i < s["sinks"] or i >= end - s["recent"]]
            sums = w[page, h, slot].tolist()
            middle = sorted(range(s["sinks"], max(s["sinks"], end - s["recent"])), key=lambda i: (-sums[i], i))
            kept = torch.tensor(sorted((forced + middle)[:count]), device="cuda")
            for t in (k, v, w):
                t[page[:count], h, slot[:count]] = t[page[kept], h, slot[kept]]
    return dict(k=k, v=v, weights=w)


def _exact_logprobs(s):
    logp = s["x"].double().log_softmax(1)
    out = dict(logprobs=logp.gather(1, s["tokens"].long()), entropy=-(logp.exp() * logp).sum(1), top_logprobs=None)
    if s["top"]:
        out["top_logprobs"] = logp.topk(s["top"], dim=1).values
    return out


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "logprobs":
        b = 2 if c["type"] == "bf16" else 4
        return {"bytes": c["N"] * (c["V"] * b + 8.0 * c["M"] + 4 + 8 * c["top"]), "flops": 4.0 * c["N"] * c["V"]}
    b, Hkv, N = 1 if c["type"] == "e4m3" else 2, c["Hkv"], c["N"]
    if c["op"] == "evict":
        # the weights are read once; kept tokens that move are read and written with their weights
        lens = (max(1, min(c["budget"], 3 * c["L"] // 4)) + c["L"]) / 2
        moved = max(0.0, min(lens, c["budget"]) - c["sinks"]) if lens > c["budget"] else 0.0
        return {"bytes": N * Hkv * (4.0 * lens + 2 * moved * (2 * D * b + 4) + 4 * c["budget"]), "flops": 0}
    tokens = c["T"] if not c["ragged"] else (max(1, c["T"] // 4) + c["T"]) / 2
    if c["op"] == "append":
        return {"bytes": N * tokens * Hkv * 2 * D * (2.0 + b), "flops": 0}
    places = c["L"] if not c["ragged"] else max((max(1, c["L"] // 3) + c["L"]) / 2, tokens)
    pairs = N * tokens * (places - (tokens - 1) / 2)
    cache = N * places * Hkv * (2.0 * D * b + (8 if c["accumulate"] else 0))
    return {"bytes": cache + N * tokens * c["Hq"] * (4.0 * D + 4), "flops": 4.0 * D * c["Hq"] * pairs}
