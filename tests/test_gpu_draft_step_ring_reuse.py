"""The decode step over drafted tokens on batches as large as a server's: every CTA of the persistent kernel
goes round its ring of stages several times. Sampled (row, head) pairs are held against the recurrence
(tolerances as derived in test_gpu_draft_step.py), and all of them, bit for bit, against the same rows
in calls so small that no stage is used twice."""
import numpy as np
import pytest
import torch

from oracle import speculative as sp

pytestmark = pytest.mark.gpu
E32, E16 = 2.0 ** -24, 2.0 ** -8
SCALE = 128 ** -0.5
STAGES = 4   # of the variant with the fewest


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_linear_attention_gb300 import build, sala_gla
    build.build()
    return sala_gla


def _tokens(gen, N, T, H, counts):
    """NaN past each row's count."""
    def unit():
        t = torch.randn(N, T, H, 128, generator=gen, device="cuda")
        return (t / t.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    q, k, v = unit(), unit(), torch.randn(N, T, H, 128, generator=gen, device="cuda").to(torch.bfloat16)
    g = torch.nn.functional.logsigmoid(2 + 4 * torch.rand(N, T, H, generator=gen, device="cuda"))
    past = torch.arange(T, device="cuda") >= counts[:, None]
    for t in (q, k, v, g):
        t[past] = float("nan")
    return q, k, v, g


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Tp", [(5, 5), (8, 1), (16, 16), (9, 12)])
def test_stages_used_many_times(sg, T, Tp, storage):
    N, H, P = 160, 32, 200
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    gen = torch.Generator(device="cuda").manual_seed(T * 100 + Tp)
    ints = lambda lo, hi: torch.randint(lo, hi, (N,), generator=gen, device="cuda", dtype=torch.int32)  # noqa: E731
    counts, accepted = ints(0, T + 1), ints(-1, Tp)
    counts[::9], accepted[4::9] = 0, -1          # rows that only commit, that only read
    slots = torch.randperm(P, generator=gen, device="cuda")[:N].to(torch.int32)
    slots[3::11] = -1
    slots[70:80] = -1                            # so many that stages hold padding items and live ones in turn
    q, k, v, g = _tokens(gen, N, T, H, counts)
    _, pk, pv, pg = _tokens(gen, N, Tp, H, accepted + 1)
    before = (0.3 * torch.randn(P, H, 128, 128, generator=gen, device="cuda")).to(storage)

    def call(pool, rows):
        s = slice(*rows)
        return sg.recurrent_draft_step(q[s], k[s], v[s], g[s], SCALE, pool, slots[s], pending=(pk[s], pv[s], pg[s]),
                                       accepted=accepted[s], num_tokens=counts[s])
    pool = before.clone()
    o = call(pool, (0, N))
    assert sg.get_device_status() == 0
    assert 2 * N * H >= 3 * 9 * sms              # three times through the longest ring
    few = STAGES * sms // (2 * H)                # rows of a call that uses a stage once at most
    pool2, o2 = before.clone(), []
    for r in range(0, N, few):
        o2.append(call(pool2, (r, min(N, r + few))))
    assert sg.get_device_status() == 0
    assert torch.equal(o, torch.cat(o2)) and torch.equal(pool, pool2)

    rng = np.random.default_rng(T)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    for n in rng.choice(N, 40, replace=False).tolist():
        slot, h, c, t = int(slots[n]), int(rng.integers(H)), int(accepted[n]) + 1, int(counts[n])
        if slot < 0:
            assert torch.all(o[n] == 0)
            continue
        tok = [f64(x[n, :, h]) for x in (q, k, v, g)]
        pend = [f64(x[n, :, h]) for x in (pk, pv, pg)]
        S = f64(before[slot, h])
        ref, kept = sp.draft_step(*tok, SCALE, S, pend, c, t)
        amag, smag = sp.draft_step(*(np.abs(x) for x in tok[:3]), tok[3], SCALE, np.abs(S),
                                   [np.abs(pend[0]), np.abs(pend[1]), pend[2]], c, t)
        G = float(np.abs(tok[3][:t]).sum() + np.abs(pend[2][:c]).sum())
        got = f64(o[n, :, h])
        assert np.all(np.abs(got - ref) <= E16 * np.abs(ref) + amag * E32 * (128 + (c + t) * (8 + G) + 16)), (n, h)
        assert np.all(got[t:] == 0)
        tol = smag * E32 * ((c + t) * (8 + G) + 16) + (E16 * np.abs(kept) if storage == torch.bfloat16 else 0)
        if c:
            assert np.all(np.abs(f64(pool[slot, h]) - kept) <= tol), (n, h)
        else:
            assert torch.equal(pool[slot, h], before[slot, h])
    idle = torch.ones(P, dtype=torch.bool, device="cuda")
    idle[slots[(slots >= 0) & (accepted >= 0)].long()] = False
    assert torch.equal(pool[idle], before[idle])
