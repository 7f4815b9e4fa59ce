"""Infinities, NaN and values near the largest of fp32 in what the decode step over drafted tokens
commits and in the states it reads. A committed state has the recurrence's infinities (with their signs)
and NaN, and is as near to it as ever elsewhere; an output is infinite or NaN where the recurrence's is.

Tolerances as derived in test_gpu_draft_step.py, on the finite places: A 2^-24 (8 n + n G + 16) for a
state, with the 128 terms of a product for o, and 2^-8 of the value for what is rounded to bf16."""
import numpy as np
import pytest
import torch

from gated_linear_attention_gb300 import inputs
from oracle import speculative as sp

pytestmark = pytest.mark.gpu
E32, E16 = 2.0 ** -24, 2.0 ** -8
INF, NAN = float("inf"), float("nan")
SCALE = 0.125


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_linear_attention_gb300 import build, sala_gla
    build.build()
    return sala_gla


def _tokens(gen, N, T, H):
    q, k = (inputs.l2_normalise(torch.randn(N, T, H, 128, generator=gen)).to(torch.bfloat16) for _ in range(2))
    v = torch.randn(N, T, H, 128, generator=gen).to(torch.bfloat16)
    return q, k, v, torch.nn.functional.logsigmoid(2 + 4 * torch.rand(N, T, H, generator=gen))


def _case(T, Tp, storage, seed):
    gen = torch.Generator().manual_seed(seed)
    c = dict(zip("qkvg", _tokens(gen, 2, T, 2)))
    c["pk"], c["pv"], c["pg"] = _tokens(gen, 2, Tp, 2)[1:]
    c["pool"] = (0.3 * torch.randn(2, 2, 128, 128, generator=gen)).to(storage)
    return c


def _check(sg, c, bad_rows=()):
    """Both rows in full. bad_rows: (n, h) whose results may hold infinities or NaN."""
    d = {n: t.cuda() for n, t in c.items()}
    N, T, H = c["q"].shape[:3]
    Tp = c["pk"].shape[1]
    o = sg.recurrent_draft_step(*(d[n] for n in "qkvg"), SCALE, d["pool"], torch.arange(N, dtype=torch.int32, device="cuda"),
                                pending=(d["pk"], d["pv"], d["pg"]) if Tp else None,
                                accepted=torch.full((N,), Tp - 1, dtype=torch.int32, device="cuda") if Tp else None).cpu()
    assert sg.get_device_status() == 0
    for n in range(N):
        for h in range(H):
            with np.errstate(all="ignore"):
                tok = [c[m][n, :, h].double().numpy() for m in "qkvg"]
                pend = [c[m][n, :, h].double().numpy() for m in ("pk", "pv", "pg")]
                S = c["pool"][n, h].double().numpy()
                ref, kept = sp.draft_step(*tok, SCALE, S, pend, Tp)
                amag, smag = sp.draft_step(*(np.abs(t) for t in tok[:3]), tok[3], SCALE, np.abs(S),
                                           [np.abs(pend[0]), np.abs(pend[1]), pend[2]], Tp)
                G = float(np.abs(tok[3]).sum() + np.abs(pend[2]).sum())
                n_tok = T + Tp
                got = d["pool"][n, h].double().cpu().numpy()
                fine = np.isfinite(kept)
                assert np.array_equal(np.isnan(got), np.isnan(kept)) and np.array_equal(np.isinf(got), np.isinf(kept))
                assert np.array_equal(got[np.isinf(kept)], kept[np.isinf(kept)])
                tol = smag * E32 * (8 * n_tok + n_tok * G + 16) + (E16 * np.abs(kept) if c["pool"].dtype == torch.bfloat16 else 0)
                assert np.all((np.abs(got - kept) <= tol)[fine])
                got = o[n, :, h].double().numpy()
                fine = np.isfinite(ref)
                assert np.array_equal(np.isfinite(got), fine)
                assert (n, h) in bad_rows or fine.all()
                tol = E16 * np.abs(ref) + amag * E32 * (128 + 8 * n_tok + n_tok * G + 16)
                assert np.all((np.abs(got - ref) <= tol)[fine])


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Tp,at", [(3, 2, 1), (5, 8, 0), (12, 16, 9), (3, 16, 15), (20, 5, 3), (2, 37, 20)])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_a_committed_value(sg, T, Tp, at, bad, storage):
    c = _case(T, Tp, storage, seed=T + Tp)
    c["pv"][1, at, 0, 77] = bad
    c["pk"][1, at, 0, 5:9] = 0.0            # 0 times an infinity is NaN
    _check(sg, c, bad_rows=((1, 0),))


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Tp,at", [(3, 2, 0), (5, 8, 7), (12, 16, 9), (20, 5, 3), (2, 37, 36)])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_a_committed_key(sg, T, Tp, at, bad, storage):
    c = _case(T, Tp, storage, seed=T + Tp)
    c["pk"][0, at, 1, 100] = bad
    c["pv"][0, at, 1, 60:70] = 0.0
    _check(sg, c, bad_rows=((0, 1),))


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Tp", [(1, 0), (6, 3), (16, 16), (33, 1)])
def test_a_stored_state(sg, T, Tp, storage):
    c = _case(T, Tp, storage, seed=T + Tp)
    c["pool"][1, 0, 3, 9], c["pool"][1, 0, 64, 9], c["pool"][1, 0, 127, 64] = INF, 1.0, NAN
    c["pool"][1, 1, 50, 20:24] = -INF
    _check(sg, c, bad_rows=((1, 0), (1, 1)))


@pytest.mark.parametrize("T,Tp", [(1, 0), (6, 3), (16, 16), (33, 1)])
def test_a_stored_state_above_the_largest_bf16(sg, T, Tp):
    # 2^128 - 2^104 and its like are finite, and so is their product with a small query
    c = _case(T, Tp, torch.float32, seed=T + Tp)
    c["pool"][0, 1, 30, 7] = torch.finfo(torch.float32).max
    c["pool"][0, 1, 90, 100] = -torch.finfo(torch.float32).max
    c["q"][0, :, 1, (30, 90)] = 2.0 ** -100
    c["pg"][0, :, 1] = 0.0
    _check(sg, c)
