"""The decode step over drafted tokens on inputs whose sums fp32 holds exactly, in any order: every
product and partial sum is a whole number of some unit, and below 2^24 of it. Outputs then differ from the
recurrence by the rounding to bf16 alone, so all comparisons are for equality, and terms that nearly
cancel in pairs leave little right of an output whose terms were cut to 17 bits on the way."""
import pytest
import torch

from oracle import speculative as sp

pytestmark = pytest.mark.gpu
SCALE = 0.125


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_linear_attention_gb300 import build, sala_gla
    build.build()
    return sala_gla


def _whole(gen, below, *shape):
    return torch.randint(-below, below + 1, shape, generator=gen).float()


def _fine_tokens(gen, N, T, H):
    """Queries, keys and values whose q . k have 20 bits: q = (1, 2^-9, 2^-18, 0 ..), k whole numbers,
    tokens 2 i and 2 i + 1 with nearly the same keys and opposite values."""
    q, k, v = (torch.zeros(N, T, H, 128) for _ in range(3))
    q[..., 0], q[..., 1], q[..., 2] = 1.0, 2.0 ** -9, 2.0 ** -18
    k[..., 0], k[..., 1], k[..., 2] = _whole(gen, 1, N, T, H), _whole(gen, 100, N, T, H), _whole(gen, 100, N, T, H)
    v[:] = 2.0 * torch.randint(0, 2, v.shape, generator=gen) - 1.0
    k[:, 1::2] = k[:, 0:T - 1:2]
    k[:, 1::2, :, 2] += _whole(gen, 3, N, T // 2, H)
    v[:, 1::2] = -v[:, 0:T - 1:2]
    return (t.to(torch.bfloat16) for t in (q, k, v))


def _check(sg, q, k, v, pool, pending=None):
    """All tokens of all rows, all pending ones committed, no gate."""
    N, T, H = q.shape[:3]
    g, d = torch.zeros(N, T, H), pool.cuda()
    kw = {}
    if pending:
        kw = dict(pending=(*(t.cuda() for t in pending), torch.zeros(pending[0].shape[:3], device="cuda")),
                  accepted=torch.full((N,), pending[0].shape[1] - 1, dtype=torch.int32, device="cuda"))
    o = sg.recurrent_draft_step(q.cuda(), k.cuda(), v.cuda(), g.cuda(), SCALE, d,
                                torch.arange(N, dtype=torch.int32, device="cuda"), **kw).cpu()
    assert sg.get_device_status() == 0
    for n in range(N):
        for h in range(H):
            tok = [t[n, :, h].double().numpy() for t in (q, k, v, g)]
            pend = [t[n, :, h].double().numpy() for t in (*pending, torch.zeros(pending[0].shape[:3]))] if pending else None
            ref, kept = sp.draft_step(*tok, SCALE, pool[n, h].double().numpy(), pend, pending[0].shape[1] if pending else 0)
            assert torch.equal(o[n, :, h], torch.from_numpy(ref).to(torch.bfloat16)), (n, h)
            assert torch.equal(d[n, h].cpu(), torch.from_numpy(kept).to(pool.dtype)), (n, h)


@pytest.mark.parametrize("T", [1, 6, 16, 37])
def test_a_state_of_24_bits(sg, T):
    # queries of -1 and 1 over four rows that nearly cancel in pairs: entries of 20 bits, sums of a few
    gen = torch.Generator().manual_seed(T)
    N, H = 2, 3
    pool = torch.zeros(N, H, 128, 128)
    half = _whole(gen, 1 << 20, N, H, 64, 128)
    pool[:, :, 0::2], pool[:, :, 1::2] = half, -half + _whole(gen, 5, N, H, 64, 128)
    q = torch.zeros(N, T, H, 64)
    at = torch.rand(N, T, H, 64, generator=gen).topk(2).indices
    q = q.scatter_(-1, at, 2.0 * torch.randint(0, 2, at.shape, generator=gen) - 1.0).repeat_interleave(2, -1)
    k, v = torch.zeros(N, T, H, 128), _whole(gen, 9, N, T, H, 128)
    _check(sg, *(t.to(torch.bfloat16) for t in (q, k, v)), pool * 2.0 ** -20)


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [2, 8, 15, 16, 40])
def test_products_with_the_new_keys_of_20_bits(sg, T, storage):
    gen = torch.Generator().manual_seed(T)
    q, k, v = _fine_tokens(gen, 2, T, 2)
    _check(sg, q, k, v, torch.zeros(2, 2, 128, 128, dtype=storage))


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Tp", [(1, 2), (5, 8), (9, 16), (3, 32)])
def test_products_with_the_pending_keys_of_20_bits(sg, T, Tp, storage):
    gen = torch.Generator().manual_seed(10 * T + Tp)
    _, pk, pv = _fine_tokens(gen, 2, Tp, 2)
    q, k, v = _fine_tokens(gen, 2, T, 2)
    _check(sg, q, torch.zeros_like(k), v, torch.zeros(2, 2, 128, 128, dtype=storage), pending=(pk, pv))
