"""Workloads of speculative decoding on Simple GLA layers and of the state pool it runs on.

Three operators, each in a plain form (elementary torch operations) and as the library's call:

verify    drafted tokens against the target's probabilities, from given random numbers
step      a decode step over several drafted tokens on pooled states, which first commits the
          tokens of the step before that were accepted
pool      copy, fork (with turnover) and compaction of the per-request states

Shapes are those of the lightning layers (32 heads of dimension 128, 24 layers, 256 sequences
on a pool of 512 slots) and odd ones around them.
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACCEPT = 0.75   # share of drafted tokens that the target accepts with the distributions below


def listed():
    return [
        # one user, four drafted tokens: latency
        dict(name="verify_one", op="verify", N=1, K=4, V=65536, type="f32", drafter=True, ragged=False),
        # a drafter without probabilities (prompt lookup): counts differ by row, odd vocabulary,
        # rows that start off 16-byte boundaries
        dict(name="verify_lookup_odd", op="verify", N=61, K=7, V=50021, type="bf16", drafter=False, ragged=True),
        # a full serving batch
        dict(name="verify_batch", op="verify", N=256, K=5, V=131072, type="f32", drafter=True, ragged=False),
        # one user, five tokens a step
        dict(name="step_one", op="step", N=1, H=32, P=16, T=5, pend=5, type="f32", ragged=False),
        # long drafts of different lengths, bf16 states, an odd batch with a padding row
        dict(name="step_ragged", op="step", N=201, H=32, P=256, T=16, pend=16, type="bf16", ragged=True),
        # a full batch on fp32 states
        dict(name="step_batch", op="step", N=256, H=32, P=512, T=5, pend=5, type="f32", ragged=False),
        # two requests' states of one layer moved to other slots
        dict(name="copy_layer", op="copy", L=1, H=32, src_slots=16, dst_slots=0, n=2, src_type="f32", dst_type="f32"),
        # prefix snapshots of all layers, kept in bf16
        dict(name="copy_snapshot", op="copy", L=24, H=32, src_slots=24, dst_slots=37, n=16, src_type="f32",
             dst_type="bf16"),
        # some requests end, new ones start from a cached prefix or from nothing; one layer
        dict(name="fork_layer", op="fork", L=1, H=32, P=64, n=6, parents=2, type="f32"),
        # beams and shared prefixes of all layers
        dict(name="fork_prefixes", op="fork", L=24, H=32, P=96, n=40, parents=5, type="bf16"),
        # one layer of a small pool with odd counts
        dict(name="compact_layer", op="compact", L=1, H=5, P=53, share=0.65, type="f32"),
        # a pool that is half empty, all layers, before it is shrunk
        dict(name="compact_pool", op="compact", L=24, H=32, P=128, share=0.5, type="bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("verify", "verify", "step", "step", "step", "copy", "fork", "compact"))
    if op == "verify":
        N, V, K = _between(rng, 1, 256), _between(rng, 4000, 131072), rng.randint(1, 8)
        while K > 1 and N * V * (K + 1) > 256 * 131072 * 6:
            K -= 1
        return dict(op=op, N=N, K=K, V=V, type=rng.choice(("f32", "bf16")), drafter=rng.random() < 0.7,
                    ragged=rng.random() < 0.5)
    if op == "step":
        H, T = rng.choice((4, 5, 8, 16, 24, 32)), rng.randint(1, 16)
        pend = rng.randint(0, 16)
        N = _between(rng, 1, max(1, min(256, 8192 * 10 // (H * (T + pend)))))
        return dict(op=op, N=N, H=H, P=N + rng.randint(0, N), T=T, pend=pend, type=rng.choice(("f32", "bf16")),
                    ragged=rng.random() < 0.5)
    L, H, P = rng.randint(1, 24), rng.choice((4, 5, 8, 16, 32)), _between(rng, 12, 96)
    if op == "copy":
        within = rng.random() < 0.5
        types = [rng.choice(("f32", "bf16"))] * 2 if within else [rng.choice(("f32", "bf16")) for _ in range(2)]
        return dict(op=op, L=L, H=H, src_slots=P, dst_slots=0 if within else _between(rng, 12, 48),
                    n=rng.randint(1, 6), src_type=types[0], dst_type=types[1])
    kind = rng.choice(("f32", "bf16"))
    if op == "fork":
        return dict(op=op, L=L, H=H, P=P, n=rng.randint(1, P // 3), parents=rng.randint(1, P // 4), type=kind)
    return dict(op=op, L=L, H=H, P=P, share=rng.choice((0.2, 0.35, 0.5, 0.65, 0.8)), type=kind)


# ---- inputs --------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"verify": _prepare_verify, "step": _prepare_step, "copy": _prepare_copy, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, gen)


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda")


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _ints(gen, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int32)


def _perm(gen, n):
    return torch.randperm(n, generator=gen, device="cuda").to(torch.int32)


def _states(gen, dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, 0.02, generator=gen)


def _prepare_verify(c, gen):
    """Softmaxes of peaked logits; the drafter's logits are the target's with noise."""
    N, K, V, dt = c["N"], c["K"], c["V"], TYPES[c["type"]]
    target = 4.0 * _randn(gen, N, K + 1, V)
    draft = (target[:, :K] + 0.7 * _randn(gen, N, K, V)).softmax(-1)
    p = target.softmax(-1).to(dt)
    del target
    if c["drafter"]:
        q = draft.to(dt)
        x = torch.multinomial(draft.reshape(N * K, V), 1, generator=gen).reshape(N, K)
    else:
        q, x = None, torch.multinomial(p[:, :K].float().reshape(N * K, V).sqrt(), 1, generator=gen).reshape(N, K)
    counts = _ints(gen, 0, K + 1, N) if c["ragged"] else None
    return dict(op="verify", p=p, q=q, x=x.to(torch.int32), u=_rand(gen, N, K), s=_rand(gen, N), counts=counts)


def _tokens(gen, n, T, H):
    """Normalised queries and keys, values, and log-decays of log-sigmoid gates."""
    def unit(t):
        return (t * torch.rsqrt((t * t).sum(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
    q, k = unit(_randn(gen, n, T, H, D)), unit(_randn(gen, n, T, H, D))
    v = _randn(gen, n, T, H, D).to(torch.bfloat16)
    g = torch.log(torch.sigmoid(2.0 + 4.0 * _rand(gen, n, T, H)))
    return q, k, v, g


def _prepare_step(c, gen):
    N, T, pend = c["N"], c["T"], c["pend"]
    q, k, v, g = _tokens(gen, N, T, c["H"])
    pending = _tokens(gen, N, pend, c["H"])[1:] if pend else None
    accepted = None
    if pend:
        accepted = _ints(gen, -1 if c["ragged"] else 0, pend, N)   # -1: nothing to commit
    counts = _ints(gen, 1, T + 1, N) if c["ragged"] else None
    slots = _perm(gen, c["P"])[:N].contiguous()
    if c["ragged"] and N > 2:
        slots[N // 2] = -1   # a padding row, as in a batch padded to a captured size
    return dict(op="step", q=q, k=k, v=v, g=g, pending=pending, accepted=accepted, counts=counts, slots=slots,
                pool=_states(gen, TYPES[c["type"]], c["P"], c["H"], D, D))


def _prepare_copy(c, gen):
    L, H, n = c["L"], c["H"], c["n"]
    src_pool = _states(gen, TYPES[c["src_type"]], L, c["src_slots"], H, D, D)
    if c["dst_slots"]:
        dst_pool = _states(gen, TYPES[c["dst_type"]], L, c["dst_slots"], H, D, D)
        src, dst = _perm(gen, c["src_slots"])[:n], _perm(gen, c["dst_slots"])[:n]
    else:
        dst_pool, order = src_pool, _perm(gen, c["src_slots"])
        src, dst = order[:n], order[n:2 * n]
    return dict(op="copy", src_pool=src_pool, dst_pool=dst_pool, src=src.contiguous(), dst=dst.contiguous())


def _prepare_fork(c, gen):
    """A full enough pool: n requests end, n start, from one of `parents` cached prefixes or,
    about one in five, from a zero state."""
    P, n = c["P"], c["n"]
    order = _perm(gen, P)
    cached, done = order[:c["parents"]], order[c["parents"]:c["parents"] + n]
    used = torch.zeros(P, dtype=torch.int32, device="cuda")
    used[order[:c["parents"] + n + (P - c["parents"] - n) // 2].long()] = 1
    parents = cached[_ints(gen, 0, c["parents"], n).long()]
    parents = torch.where(_rand(gen, n) < 0.2, torch.full_like(parents, -1), parents)
    return dict(op="fork", pool=_states(gen, TYPES[c["type"]], c["L"], P, c["H"], D, D), used=used,
                done=done.contiguous(), parents=parents.contiguous())


def _prepare_compact(c, gen):
    used = (_rand(gen, c["P"]) < c["share"]).to(torch.int32)
    return dict(op="compact", pool=_states(gen, TYPES[c["type"]], c["L"], c["P"], c["H"], D, D), used=used)


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"verify": _plain_verify, "step": _plain_step, "copy": _plain_copy, "fork": _plain_fork,
            "compact": _plain_compact}[state["op"]](state)


def _run_own(s):
    from gated_linear_attention_gb300 import sala_gla
    if s["op"] == "verify":
        tokens, accepted = sala_gla.verify_drafts(s["p"], s["q"], s["x"], s["u"], s["s"], num_drafts=s["counts"])
        return dict(tokens=tokens, accepted=accepted)
    if s["op"] == "step":
        o = sala_gla.recurrent_draft_step(s["q"], s["k"], s["v"], s["g"], SCALE, s["pool"], s["slots"],
                                          pending=s["pending"], accepted=s["accepted"], num_tokens=s["counts"])
        return dict(o=o, pool=s["pool"])
    if s["op"] == "copy":
        sala_gla.state_pool_copy(s["dst_pool"], s["src_pool"], s["dst"], s["src"])
        return dict(pool=s["dst_pool"])
    used = s["used"].clone()
    if s["op"] == "fork":
        sala_gla.state_pool_free(used, s["done"])
        children = sala_gla.state_pool_fork(s["pool"], used, s["parents"])
        return dict(pool=s["pool"], used=used, children=children)
    mapping, live = sala_gla.state_pool_compact(s["pool"], used)
    return dict(pool=s["pool"], used=used, mapping=mapping, live=live)


def _plain_verify(s):
    p, q, x, u, draw_at = s["p"], s["q"], s["x"].long(), s["u"], s["s"]
    N, K = x.shape
    # the test lies next to a border, and so does the draw from the cumulative sums: 64 bits
    px = p[:, :K].gather(2, x[:, :, None])[:, :, 0].double()
    qx = q.gather(2, x[:, :, None])[:, :, 0].double() if q is not None else torch.ones_like(px)
    place = torch.arange(K, device=x.device)
    drafts = s["counts"].long() if s["counts"] is not None else torch.full((N,), K, device=x.device)
    ok = (u.double() * qx < px) & (place < drafts[:, None])
    accepted = ok.long().cumprod(1).sum(1)
    rows = torch.arange(N, device=x.device)
    target = p[rows, accepted].double()
    at = accepted.clamp(max=K - 1)
    if q is not None:
        less = q[rows, at].double()
    else:
        less = torch.zeros_like(target).scatter_(1, x[rows, at][:, None], 1.0)
    rest = (target - less).clamp(min=0)
    rest = torch.where(((accepted < drafts) & (rest.sum(1) > 0))[:, None], rest, target)
    sums = rest.cumsum(1)
    token = (sums <= draw_at.double()[:, None] * sums[:, -1:]).sum(1)
    place = torch.arange(K + 1, device=x.device)
    drafted = torch.nn.functional.pad(x, (0, 1))
    tokens = torch.where(place < accepted[:, None], drafted, torch.full_like(drafted, -1))
    tokens = torch.where(place == accepted[:, None], token[:, None], tokens)
    return dict(tokens=tokens.to(torch.int32), accepted=accepted.to(torch.int32))


def _plain_step(s):
    pool, slots = s["pool"], s["slots"]
    live = slots >= 0
    at = slots.clamp(min=0).long()
    S = pool[at].float()
    if s["pending"] is not None:
        pk, pv, pg = (t.float() for t in s["pending"])
        kept = (torch.arange(pk.shape[1], device=pk.device) <= s["accepted"][:, None])[:, :, None]
        G = torch.where(kept, pg, torch.zeros_like(pg)).cumsum(1)
        w = torch.where(kept, (G[:, -1:] - G).exp(), torch.zeros_like(G))
        S = G[:, -1].exp()[:, :, None, None] * S + torch.matmul((pk * w[..., None]).permute(0, 2, 3, 1),
                                                                pv.permute(0, 2, 1, 3))
        pool[at[live]] = S[live].to(pool.dtype)
    q, k, v = (s[n].float().permute(0, 2, 1, 3) for n in ("q", "k", "v"))   # [N, H, T, 128]
    G = s["g"].permute(0, 2, 1).cumsum(2)
    T = G.shape[2]
    before = torch.ones(T, T, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(before, G[..., :, None] - G[..., None, :], torch.full((), -math.inf, device=q.device)).exp()
    o = torch.matmul(q, S) * G.exp()[..., None] + torch.matmul(torch.matmul(q, k.transpose(2, 3)) * decay, v)
    o = (SCALE * o).permute(0, 2, 1, 3)
    if s["counts"] is not None:
        live = live[:, None] & (torch.arange(T, device=q.device) < s["counts"][:, None])
    else:
        live = live[:, None].expand(-1, T)
    o = torch.where(live[:, :, None, None], o, torch.zeros_like(o))
    return dict(o=o.to(torch.bfloat16).contiguous(), pool=pool)


def _plain_copy(s):
    s["dst_pool"][:, s["dst"].long()] = s["src_pool"][:, s["src"].long()].to(s["dst_pool"].dtype)
    return dict(pool=s["dst_pool"])


def _plain_fork(s):
    pool, used, parents = s["pool"], s["used"].clone(), s["parents"].long()
    used[s["done"].long()] = 0
    children = (used == 0).nonzero()[:, 0][:parents.numel()]
    used[children] = 1
    old = parents >= 0
    pool[:, children[old]] = pool[:, parents[old]]
    pool[:, children[~old]] = 0
    return dict(pool=pool, used=used, children=children.to(torch.int32))


def _plain_compact(s):
    pool, used = s["pool"], s["used"].clone()
    P = used.numel()
    live = used.sum()
    slot = torch.arange(P, device=used.device)
    src = ((used != 0) & (slot >= live)).nonzero()[:, 0]
    dst = ((used == 0) & (slot < live)).nonzero()[:, 0]
    mapping = torch.where(used != 0, slot, torch.full_like(slot, -1))
    mapping[src] = dst
    pool[:, dst] = pool[:, src]
    used = (slot < live).to(torch.int32)
    return dict(pool=pool, used=used, mapping=mapping.to(torch.int32), live=live.to(torch.int32).reshape(1))


# ---- the definition in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "step":
        return _exact_step(s)
    if case["op"] == "verify":
        return None     # whole numbers only
    if case["op"] == "copy":
        pool = s["dst_pool"].double()
        for i, j in zip(s["src"].tolist(), s["dst"].tolist()):
            pool[:, j] = s["src_pool"][:, i].double()
        return dict(pool=pool)
    return dict(pool=_moved(s))


def _moved(s):
    """The pool after a fork or a compaction, slot by slot (values move, none is computed)."""
    pool, used = s["pool"], s["used"].tolist()
    if s["op"] == "fork":
        for i in s["done"].tolist():
            used[i] = 0
        for parent in s["parents"].tolist():
            child = used.index(0)
            used[child] = 1
            pool[:, child] = pool[:, parent] if parent >= 0 else 0
        return pool
    live = sum(1 for x in used if x)
    holes = iter([i for i in range(live) if not used[i]])
    for i in range(live, len(used)):
        if used[i]:
            pool[:, next(holes)] = pool[:, i]
    return pool


def _exact_step(s):
    """The recurrence token by token, one row of the batch at a time."""
    N, T, H, _ = s["q"].shape
    pool = s["pool"].double()
    o = torch.zeros(N, T, H, D, dtype=torch.float64, device="cuda")
    accepted = s["accepted"].tolist() if s["accepted"] is not None else [-1] * N
    counts = s["counts"].tolist() if s["counts"] is not None else [T] * N
    for n, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        S = pool[slot].clone()
        for j in range(accepted[n] + 1):
            k, v, g = (t[n, j].double() for t in s["pending"])
            S = g.exp()[:, None, None] * S + k[:, :, None] * v[:, None, :]
        pool[slot] = S
        for t in range(counts[n]):
            S = s["g"][n, t].double().exp()[:, None, None] * S
            S = S + s["k"][n, t].double()[:, :, None] * s["v"][n, t].double()[:, None, :]
            o[n, t] = SCALE * (s["q"][n, t].double()[:, :, None] * S).sum(1)
    return dict(o=o, pool=pool)


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "verify":
        N, K, V, b = c["N"], c["K"], c["V"], 2 if c["type"] == "bf16" else 4
        lengths = range(K + 1) if c["ragged"] else (K,)
        rejected = sum(1.0 - ACCEPT ** k for k in lengths) / len(lengths)
        rows = 1.0 + (rejected if c["drafter"] else 0.0)   # the drafter's row only where a token was rejected
        return {"bytes": N * (rows * V * b + 12.0 * K + 8 * b * K + 4 * (K + 3)), "flops": 4.0 * N * V}
    if c["op"] == "step":
        N, H, T, pend, b = c["N"], c["H"], c["T"], c["pend"], 2 if c["type"] == "bf16" else 4
        commits = (pend + 1) / 2 if pend else 0
        tokens = (T + 1) / 2 if c["ragged"] else T
        states = N * H * D * D * b * (2 if pend else 1)
        vectors = N * H * D * 2 * (3 * tokens + T + 2 * commits) + N * H * 4 * (tokens + commits)
        return {"bytes": states + vectors, "flops": 2.0 * N * H * D * D * (tokens + commits)}
    slot = c["L"] * c["H"] * D * D
    if c["op"] == "copy":
        return {"bytes": c["n"] * slot * sum(2 if c[t] == "bf16" else 4 for t in ("src_type", "dst_type")), "flops": 0}
    slot *= 2 if c["type"] == "bf16" else 4
    if c["op"] == "fork":
        return {"bytes": slot * (min(c["parents"], 0.8 * c["n"]) + c["n"]) + 8 * c["P"], "flops": 0}
    moves = c["P"] * c["share"] * (1 - c["share"])
    return {"bytes": 2 * slot * moves + 12 * c["P"], "flops": 0}
