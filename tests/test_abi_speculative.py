"""Host-side checks of the speculative-decoding and state-pool entry points (no GPU needed): bad
arguments are refused before CUDA is touched, valid ones then report that there is no device."""
import ctypes

import pytest
import torch

from gated_linear_attention_gb300 import build as B

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake pointers must never reach a real device")
P = ctypes.c_void_p
INVALID, MISALIGNED, CUDA = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    B.build()
    from gated_linear_attention_gb300 import sala_gla
    return sala_gla.load()


def _p(x):
    return P(x) if x else None


def _verify(lib, p=0x100000, pld=1000, q=0x200000, qld=1000, dt=0, x=0x300000, nd=None, u=0x310000,
            s=0x320000, tok=0x330000, acc=0x340000, N=2, K=3, V=1000):
    return lib.sala_gla_verify_drafts(_p(p), pld, _p(q), qld, dt, _p(x), _p(nd), _p(u), _p(s), _p(tok),
                                      _p(acc), N, K, V, None)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(V=0), INVALID), (dict(V=(1 << 20) + 1), INVALID),
    (dict(dt=2), INVALID), (dict(pld=999), INVALID), (dict(qld=999), INVALID), (dict(p=0), INVALID),
    (dict(x=0), INVALID), (dict(u=0), INVALID), (dict(s=0), INVALID), (dict(tok=0), INVALID),
    (dict(acc=0), INVALID), (dict(p=0x100002), MISALIGNED), (dict(q=0x200001, dt=1), MISALIGNED),
    (dict(x=0x300002), MISALIGNED), (dict(tok=0x330001), MISALIGNED), (dict(nd=0x350002), MISALIGNED),
    (dict(tok=0x100000 + 4), INVALID), (dict(acc=0x330000 + 4), INVALID), (dict(acc=0x310000), INVALID),
    (dict(N=0), 0), (dict(p=0x100002, dt=1), CUDA), (dict(q=0), CUDA), (dict(nd=0x350004), CUDA),
    (dict(K=0, x=0, u=0, q=0), CUDA), (dict(pld=1 << 33), INVALID), (dict(), CUDA)])
def test_verify_drafts_argument_errors(lib, kw, want):
    assert _verify(lib, **kw) == want


def _step(lib, q=0x100000, k=0x110000, v=0x120000, g=0x130000, nt=None, pk=0x140000, pv=0x150000,
          pg=0x160000, acc=0x170000, pool=0x1000000, dt=0, idx=0x180000, Pn=4, o=0x190000, N=2, T=3, Tp=3,
          H=2):
    return lib.sala_gla_recurrent_draft_step(_p(q), _p(k), _p(v), _p(g), _p(nt), _p(pk), _p(pv), _p(pg),
                                             _p(acc), 0.1, _p(pool), dt, _p(idx), Pn, _p(o), N, T, Tp, H,
                                             None)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(Tp=-1), INVALID), (dict(H=0), INVALID),
    (dict(Pn=0), INVALID), (dict(dt=2), INVALID), (dict(pool=0), INVALID), (dict(idx=0), INVALID),
    (dict(q=0), INVALID), (dict(o=0), INVALID), (dict(pk=0), INVALID), (dict(pg=0), INVALID),
    (dict(acc=0), INVALID), (dict(N=1 << 31), INVALID), (dict(q=0x100008), MISALIGNED),
    (dict(o=0x190008), MISALIGNED), (dict(pv=0x150002), MISALIGNED), (dict(pool=0x1000008), MISALIGNED),
    (dict(g=0x130002), MISALIGNED), (dict(acc=0x170001), MISALIGNED), (dict(idx=0x180002), MISALIGNED),
    (dict(nt=0x1a0001), MISALIGNED), (dict(o=0x100000 + 16), INVALID), (dict(o=0x1000000 + 4096), INVALID),
    (dict(pool=0x160000), INVALID), (dict(idx=0x1000000 + 64), INVALID),
    (dict(N=0), 0), (dict(T=0, Tp=0), 0), (dict(g=0x130004), CUDA),
    (dict(T=0, q=0, k=0, v=0, g=0, o=0), CUDA), (dict(Tp=0, pk=0, pv=0, pg=0, acc=0), CUDA),
    (dict(dt=1), CUDA), (dict(), CUDA)])
def test_draft_step_argument_errors(lib, kw, want):
    assert _step(lib, **kw) == want


def _copy(lib, sp=0x10000000, sd=0, sP=4, dp=0x20000000, dd=1, dP=5, src=0x1000, dst=0x2000, n=3, L=2, H=2):
    return lib.sala_gla_state_pool_copy(_p(sp), sd, sP, _p(dp), dd, dP, _p(src), _p(dst), n, L, H, None)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(sp=0), INVALID), (dict(dp=0), INVALID), (dict(sd=2), INVALID), (dict(dd=-1), INVALID),
    (dict(sP=0), INVALID), (dict(dP=0), INVALID), (dict(L=0), INVALID), (dict(H=0), INVALID),
    (dict(n=-1), INVALID), (dict(src=0), INVALID), (dict(dst=0), INVALID),
    (dict(dp=0x10000000, dd=1, dP=4), INVALID),        # one pool, two types
    (dict(dp=0x10000000, dd=0, dP=5), INVALID),        # one pool, two sizes
    (dict(dp=0x10000000 + 65536), INVALID),            # pools overlap in part
    (dict(dst=0x20000000 + 64), INVALID),              # slots inside the destination
    (dict(sp=0x10000008), MISALIGNED), (dict(src=0x1002), MISALIGNED),
    (dict(n=0, src=0, dst=0), 0), (dict(dp=0x10000000, dd=0, dP=4), CUDA), (dict(), CUDA)])
def test_state_pool_copy_argument_errors(lib, kw, want):
    assert _copy(lib, **kw) == want


def _fork(lib, pool=0x10000000, dt=0, L=2, Pn=8, H=2, used=0x1000, par=0x2000, kid=0x3000, n=3):
    return lib.sala_gla_state_pool_fork(_p(pool), dt, L, Pn, H, _p(used), _p(par), _p(kid), n, None)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(pool=0), INVALID), (dict(dt=7), INVALID), (dict(Pn=0), INVALID), (dict(n=-1), INVALID),
    (dict(used=0), INVALID), (dict(par=0), INVALID), (dict(kid=0), INVALID), (dict(kid=0x2004), INVALID),
    (dict(used=0x2004), INVALID), (dict(kid=0x1010), INVALID), (dict(used=0x10000040), INVALID),
    (dict(kid=0x3001), MISALIGNED), (dict(pool=0x10000004), MISALIGNED), (dict(n=0), 0), (dict(), CUDA)])
def test_state_pool_fork_argument_errors(lib, kw, want):
    assert _fork(lib, **kw) == want


@no_gpu
@pytest.mark.parametrize("args,want", [
    ((0x1000, 0, 0x2000, 3), INVALID), ((0x1000, 8, 0x2000, -1), INVALID), ((0, 8, 0x2000, 3), INVALID),
    ((0x1000, 8, 0, 3), INVALID), ((0x1000, 8, 0x101c, 3), INVALID), ((0x1002, 8, 0x2000, 3), MISALIGNED),
    ((0x1000, 8, 0, 0), 0), ((0x1000, 8, 0x2000, 3), CUDA)])
def test_state_pool_free_argument_errors(lib, args, want):
    used, Pn, slots, n = args
    assert lib.sala_gla_state_pool_free(_p(used), Pn, _p(slots), n, None) == want


def _compact(lib, pool=0x10000000, dt=0, L=2, Pn=8, H=2, used=0x1000, m=0x2000, live=0x3000):
    return lib.sala_gla_state_pool_compact(_p(pool), dt, L, Pn, H, _p(used), _p(m), _p(live), None)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(pool=0), INVALID), (dict(used=0), INVALID), (dict(m=0), INVALID), (dict(live=0), INVALID),
    (dict(m=0x1004), INVALID), (dict(live=0x2008), INVALID), (dict(live=0x10000000), INVALID),
    (dict(H=0), INVALID), (dict(live=0x4002), MISALIGNED), (dict(), CUDA)])
def test_state_pool_compact_argument_errors(lib, kw, want):
    assert _compact(lib, **kw) == want


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    from gated_linear_attention_gb300 import sala_gla as sg
    p, i2 = torch.zeros(2, 4, 50), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        sg.verify_drafts(p, None, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(2))
    with pytest.raises(ValueError):
        sg.verify_drafts(p[0], None, i2, i2, i2)
    with pytest.raises(TypeError):
        sg.verify_drafts(p.double(), None, i2, i2, i2)
    pool = torch.zeros(4, 1, 128, 128)
    for call in (lambda: sg.recurrent_draft_step(None, None, None, None, 0.1, pool, i2),
                 lambda: sg.state_pool_copy(pool, pool, i2, i2), lambda: sg.state_pool_fork(pool, i2, i2),
                 lambda: sg.state_pool_free(i2, i2), lambda: sg.state_pool_compact(pool, i2)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        sg.state_pool_compact(pool.double(), i2)
