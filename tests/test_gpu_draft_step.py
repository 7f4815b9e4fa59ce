"""The decode step over drafted tokens (sala_gla_recurrent_draft_step) against the recurrence in
fp64, token by token.

Tolerances, per element. Let A be the sum of the magnitudes of the terms of an element (the
recurrence run on |q|, |k|, |v|, |S|), n the number of tokens that reach it and G the magnitude of
their summed gates. In fp32 a chain of 128 products and their sums, the n decayed terms and the
exponentials (of sums of up to n gates, each sum off by n 2^-24 G, the function by 2 ulp) stay within
    A 2^-24 (128 + 8 n + n G + 16)
for o, and without the 128 for a state. A bf16 result adds half a step, 2^-8 of its value.
"""
import numpy as np
import pytest
import torch

from gated_linear_attention_gb300 import inputs
from oracle import speculative as sp

pytestmark = pytest.mark.gpu
E32, E16 = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_linear_attention_gb300 import build, sala_gla
    build.build()
    return sala_gla


def _tokens(gen, N, T, H, gate):
    q, k = (inputs.l2_normalise(torch.randn(N, T, H, 128, generator=gen)).to(torch.bfloat16) for _ in range(2))
    v = torch.randn(N, T, H, 128, generator=gen).to(torch.bfloat16)
    if gate == "mild":
        g = torch.nn.functional.logsigmoid(2 + 4 * torch.rand(N, T, H, generator=gen))
    else:                                   # forget nothing, something, everything, and grow
        g = torch.tensor([0.0, -0.5, -30.0, float("-inf"), 0.25])[torch.randint(0, 5, (N, T, H), generator=gen)]
    return q, k, v, g


def _case(N, T, Tp, H, P, storage, seed, gate="mild", ragged=True, pad=()):
    gen = torch.Generator().manual_seed(seed)
    q, k, v, g = _tokens(gen, N, T, H, gate)
    _, pk, pv, pg = _tokens(gen, N, Tp, H, gate)
    pool = (0.3 * torch.randn(P, H, 128, 128, generator=gen)).to(storage)
    slots = torch.randperm(P, generator=gen)[:N].to(torch.int32)
    for r in pad:
        slots[r] = -1
    accepted = torch.randint(-1, Tp, (N,), generator=gen, dtype=torch.int32) if Tp else None
    counts = torch.randint(0, T + 1, (N,), generator=gen, dtype=torch.int32) if ragged and T else None
    if not ragged and Tp:
        accepted[:] = Tp - 1
    return dict(q=q, k=k, v=v, g=g, pending=(pk, pv, pg) if Tp else None, accepted=accepted, counts=counts,
                pool=pool, slots=slots)


def _run(sg, c, scale, **kw):
    cu = lambda t: t.cuda() if t is not None else None  # noqa: E731
    pool = c["pool"].cuda()
    T = c["q"].shape[1]
    tok = [cu(c[n]) for n in ("q", "k", "v", "g")] if T else [None] * 4
    o = sg.recurrent_draft_step(*tok, scale, pool, cu(c["slots"]),
                                pending=tuple(cu(t) for t in c["pending"]) if c["pending"] else None,
                                accepted=cu(c["accepted"]), num_tokens=cu(c["counts"]) if T else None, **kw)
    torch.cuda.synchronize()
    return (o.cpu() if o is not None else None), pool.cpu()


def _sum_gates(g):
    g = np.asarray(g, np.float64)
    return float(np.abs(g[np.isfinite(g)]).sum())


def _check(c, o, pool, scale, only=None):
    P, H = c["pool"].shape[:2]
    N, T = c["q"].shape[:2]
    touched = set()
    for n in range(N):
        slot = int(c["slots"][n])
        if slot < 0:
            assert o is None or torch.all(o[n] == 0)
            continue
        commits = int(c["accepted"][n]) + 1 if c["accepted"] is not None else 0
        count = int(c["counts"][n]) if c["counts"] is not None else T
        if commits:
            touched.add(slot)
        for h in (range(H) if only is None else only):
            tok = [c[m][n, :, h].double().numpy() for m in ("q", "k", "v", "g")]
            pend = [t[n, :, h].double().numpy() for t in c["pending"]] if c["pending"] else None
            S = c["pool"][slot, h].double().numpy()
            ref, kept = sp.draft_step(*tok, scale, S, pend, commits, count)
            mag = [np.abs(x) for x in tok[:3]] + [tok[3]]
            amag, smag = sp.draft_step(*mag, scale, np.abs(S),
                                       [np.abs(pend[0]), np.abs(pend[1]), pend[2]] if pend else None, commits, count)
            G = _sum_gates(tok[3][:count]) + (_sum_gates(pend[2][:commits]) if pend else 0.0)
            n_tok = commits + count
            if commits:
                tol = smag * E32 * (8 * n_tok + n_tok * G + 16) + (E16 * np.abs(kept) if c["pool"].dtype == torch.bfloat16 else 0)
                got = pool[slot, h].double().numpy()
                assert np.all(np.abs(got - kept) <= tol), (n, h, np.abs(got - kept).max())
            if o is not None:
                got = o[n, :, h].double().numpy()
                tol = E16 * np.abs(ref) + amag * E32 * (128 + 8 * n_tok + n_tok * G + 16)
                assert np.all(np.abs(got - ref) <= tol), (n, h, np.abs(got - ref).max())
                assert np.all(got[count:] == 0)
    others = [s for s in range(P) if s not in touched]
    assert torch.equal(pool[others], c["pool"][others])


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,T,Tp,H,P", [(1, 1, 0, 1, 1), (1, 1, 1, 1, 2), (3, 5, 5, 2, 4), (2, 8, 3, 3, 5),
                                        (2, 9, 17, 1, 3), (1, 16, 16, 2, 1), (1, 33, 0, 1, 1), (2, 0, 6, 2, 3),
                                        (1, 70, 41, 1, 1), (40, 3, 4, 5, 64)])
@pytest.mark.parametrize("gate", ["mild", "wild"])
def test_against_the_recurrence(sg, N, T, Tp, H, P, storage, gate):
    c = _case(N, T, Tp, H, P, storage, seed=N + 10 * T + 100 * Tp, gate=gate, pad=(0,) if N > 2 else ())
    o, pool = _run(sg, c, 128 ** -0.5)
    assert sg.get_device_status() == 0
    _check(c, o, pool, 128 ** -0.5)


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
def test_full_counts(sg, storage):
    c = _case(4, 6, 6, 4, 9, storage, seed=77, ragged=False)
    o, pool = _run(sg, c, 0.125)
    _check(c, o, pool, 0.125)


def test_nothing_pending_leaves_the_pool(sg):
    c = _case(3, 4, 0, 2, 4, torch.bfloat16, seed=5, ragged=False)
    o, pool = _run(sg, c, 0.125)
    assert torch.equal(pool, c["pool"])
    c2 = _case(3, 4, 4, 2, 4, torch.float32, seed=6, ragged=False)
    c2["accepted"][:] = -1
    _, pool = _run(sg, c2, 0.125)
    assert torch.equal(pool, c2["pool"])


def test_one_call_equals_commit_then_step(sg):
    # fp32 states: committing in one call and stepping in the next gives the same bits
    c = _case(5, 7, 6, 3, 8, torch.float32, seed=15, ragged=True)
    o, pool = _run(sg, c, 0.125)
    commit = dict(c, q=c["q"][:, :0], k=c["k"][:, :0], v=c["v"][:, :0], g=c["g"][:, :0])
    none, pool2 = _run(sg, commit, 0.125)
    assert none is None and torch.equal(pool, pool2)
    step = dict(c, pool=pool2, pending=None, accepted=None)
    o2, pool3 = _run(sg, step, 0.125)
    assert torch.equal(pool3, pool2) and torch.equal(o, o2)


def test_agrees_with_the_one_token_step(sg):
    # a chain of draft steps that accept everything against the pooled one-token decode
    c = _case(4, 5, 0, 2, 6, torch.float32, seed=31, ragged=False)
    o, _ = _run(sg, c, 0.125)
    pool = c["pool"].cuda()
    for t in range(5):
        ref = sg.recurrent_step_indexed(*(c[n][:, t].contiguous().cuda() for n in ("q", "k", "v", "g")), 0.125,
                                        pool, c["slots"].cuda()).cpu()
        assert (o[:, t].double() - ref.double()).abs().max() <= 2 * E16 * ref.double().abs().max()
    commit = dict(c, q=c["q"][:, :0], pending=(c["k"], c["v"], c["g"]), accepted=torch.full((4,), 4, dtype=torch.int32),
                  counts=None)
    _, kept = _run(sg, commit, 0.125)
    assert (kept - pool.cpu()).abs().max() <= 1e-5


@pytest.mark.parametrize("what", ["slot", "accepted", "count", "negative count"])
def test_rows_outside_their_range_are_reported_and_skipped(sg, what):
    c = _case(4, 3, 3, 2, 6, torch.float32, seed=41, ragged=False)
    c["counts"] = torch.full((4,), 3, dtype=torch.int32)
    if what == "slot":
        c["slots"][2] = 6
    elif what == "accepted":
        c["accepted"][2] = 3
    else:
        c["counts"][2] = 4 if what == "count" else -1
    o, pool = _run(sg, c, 0.125)
    assert sg.get_device_status() == 8 and sg.get_device_status() == 0
    assert torch.all(o[2] == 0)
    c["slots"][2] = -1
    _check(dict(c, counts=None), o, pool, 0.125)


def test_far_slots_of_a_large_pool(sg):
    # offsets past 2^32 bytes and 2^31 elements: 2100 slots of 32 heads in bf16 (2.2 GB) and a batch
    # on its first and last slots
    c = _case(3, 2, 2, 32, 4, torch.bfloat16, seed=51, ragged=False)
    big = torch.zeros(2 ** 31 // (32 * 128 * 128) + 52, 32, 128, 128, dtype=torch.bfloat16, device="cuda")
    far = torch.tensor([0, big.shape[0] - 1, big.shape[0] // 2 + 1])
    here = c["slots"].long()
    big[far.cuda()] = c["pool"][here].cuda()
    tok = [c[n].cuda() for n in ("q", "k", "v", "g")]
    o = sg.recurrent_draft_step(*tok, 0.125, big, far.to(torch.int32).cuda(),
                                pending=tuple(t.cuda() for t in c["pending"]), accepted=c["accepted"].cuda()).cpu()
    pool = c["pool"].clone()
    pool[here] = big[far.cuda()].cpu()
    assert sg.get_device_status() == 0
    _check(c, o, pool, 0.125, only=(0, 31))
    assert int((big != 0).any(dim=(1, 2, 3)).sum()) == 3


def test_graph_and_side_stream(sg):
    c = _case(6, 4, 4, 3, 9, torch.bfloat16, seed=61)
    d = {n: c[n].cuda() for n in ("q", "k", "v", "g", "slots", "accepted", "counts", "pool")}
    pend = tuple(t.cuda() for t in c["pending"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = sg.recurrent_draft_step(d["q"], d["k"], d["v"], d["g"], 0.125, d["pool"], d["slots"], pending=pend,
                                accepted=d["accepted"], num_tokens=d["counts"], stream=side)
    side.synchronize()
    _check(c, o.cpu(), d["pool"].cpu(), 0.125)
    d["pool"].copy_(c["pool"])
    out = torch.empty_like(d["q"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.recurrent_draft_step(d["q"], d["k"], d["v"], d["g"], 0.125, d["pool"], d["slots"], pending=pend,
                                accepted=d["accepted"], num_tokens=d["counts"], o=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), o.cpu())
    _check(c, out.cpu(), d["pool"].cpu(), 0.125)


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Tp", [(5, 5), (8, 3), (13, 16), (20, 19)])
def test_masked_places_hold_anything(sg, T, Tp, storage):
    # NaN in tokens past the counts (and in their gates) changes nothing
    c = _case(6, T, Tp, 2, 9, storage, seed=T + Tp)
    c["accepted"][0], c["counts"][0] = -1, 0
    o, pool = _run(sg, c, 0.125)
    for n in range(6):
        for t in c["pending"]:
            t[n, int(c["accepted"][n]) + 1:] = float("nan")
        for name in ("q", "k", "v", "g"):
            c[name][n, int(c["counts"][n]):] = float("nan")
    o2, pool2 = _run(sg, c, 0.125)
    assert torch.equal(o, o2) and torch.equal(pool, pool2)


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,at", [(6, 3), (16, 11), (12, 0)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_bad_value_reaches_only_the_tokens_from_its_own_on(sg, T, at, bad, storage):
    c = _case(2, T, 2, 2, 3, storage, seed=T, ragged=False)
    o, pool = _run(sg, c, 0.125)
    c["v"][1, at, 0, 77] = bad
    o2, pool2 = _run(sg, c, 0.125)
    assert torch.equal(pool, pool2)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[1, at:, 0, 77] = True
    assert not o2[hit].isfinite().any()
    near = (o.double() - o2.double()).abs() <= 2 * E16 * o.double().abs() + 1e-6
    assert torch.all(near | hit)


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Tp", [(17, 1), (1, 17), (31, 32), (33, 47), (48, 16), (0, 40), (16, 64)])
def test_counts_around_the_edges_of_longer_steps(sg, T, Tp, storage):
    # more than 16 tokens go over the state in blocks: counts at, before and after a block's end
    c = _case(6, T, Tp, 2, 8, storage, seed=900 + T + 100 * Tp, gate="wild", pad=(1,))
    for n, x in enumerate((0, 0, 15, 16, 17, 33)):
        c["accepted"][n] = min(x, Tp) - 1
        if T:
            c["counts"][5 - n] = min(x, T)
    o, pool = _run(sg, c, 0.125)
    assert sg.get_device_status() == 0
    _check(c, o, pool, 0.125)


def test_a_longer_call_equals_commit_then_step(sg):
    c = _case(4, 37, 35, 2, 6, torch.float32, seed=71, ragged=True)
    o, pool = _run(sg, c, 0.125)
    commit = dict(c, q=c["q"][:, :0], k=c["k"][:, :0], v=c["v"][:, :0], g=c["g"][:, :0])
    none, pool2 = _run(sg, commit, 0.125)
    assert none is None and torch.equal(pool, pool2)
    o2, pool3 = _run(sg, dict(c, pool=pool2, pending=None, accepted=None), 0.125)
    assert torch.equal(pool3, pool2) and torch.equal(o, o2)


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [3, 16, 20, 39])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_bad_value_of_a_longer_step(sg, at, bad, storage):
    c = _case(2, 40, 2, 2, 3, storage, seed=at, ragged=False)
    o, pool = _run(sg, c, 0.125)
    c["v"][1, at, 0, 77] = bad
    o2, pool2 = _run(sg, c, 0.125)
    assert torch.equal(pool, pool2)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[1, at:, 0, 77] = True
    assert not o2[hit].isfinite().any()
    near = (o.double() - o2.double()).abs() <= 2 * E16 * o.double().abs() + 1e-6
    assert torch.all(near | hit)
