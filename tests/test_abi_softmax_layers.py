"""Host-side checks of the softmax layers' entry points (no GPU needed): bad arguments are refused before CUDA
is touched, valid ones then report that there is no device."""
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


def _cache(kp=0x10000000, vp=0x20000000, ks=0, vs=0, w=0x30000000, table=0x1000, lens=0x2000, pages=8, width=4, page=16,
           H=2, dt=0):
    from gated_linear_attention_gb300.sala_gla import KvCacheStruct
    return KvCacheStruct(kp or None, vp or None, ks or None, vs or None, w or None, table or None, lens or None, pages,
                         width, page, H, dt)


CACHE_CASES = [
    (dict(kp=0), INVALID), (dict(vp=0), INVALID), (dict(table=0), INVALID), (dict(lens=0), INVALID),
    (dict(page=8), INVALID), (dict(page=48), INVALID), (dict(page=512), INVALID), (dict(page=0), INVALID),
    (dict(H=0), INVALID), (dict(H=65536), INVALID), (dict(pages=0), INVALID), (dict(width=0), INVALID),
    (dict(pages=1 << 31), INVALID), (dict(width=1 << 28), INVALID), (dict(dt=2), INVALID), (dict(ks=0x5000), INVALID),
    (dict(vs=0x5000), INVALID), (dict(kp=0x10000008), MISALIGNED), (dict(vp=0x20000004), MISALIGNED),
    (dict(w=0x30000002), MISALIGNED), (dict(table=0x1002), MISALIGNED), (dict(lens=0x2001), MISALIGNED),
    (dict(dt=1, ks=0x5002), MISALIGNED), (dict(vp=0x10000100), INVALID), (dict(w=0x10000100), INVALID),
    (dict(table=0x10000100), INVALID), (dict(lens=0x20000100), INVALID), (dict(dt=1, ks=0x20000100), INVALID),
    (dict(dt=1, ks=0x5000, vs=0x6000), CUDA), (dict(page=256), CUDA), (dict(), CUDA)]


def _append(lib, k=0x100000, kld=256, v=0x200000, vld=256, cu=0x3000, N=3, T=5, **cache):
    c = _cache(**cache)
    return lib.sala_gla_kv_append(ctypes.byref(c), _p(k), kld, _p(v), vld, _p(cu), N, T, None)


def _attend(lib, q=0x100000, ld=4096, scale=0.1, cu=0x3000, o=0x400000, lse=0x500000, acc=1, N=3, T=5, Hq=32, **cache):
    c = _cache(**cache)
    return lib.sala_gla_paged_attention(ctypes.byref(c), _p(q), ld, scale, _p(cu), _p(o), _p(lse), acc, N, T, Hq, None)


def _evict(lib, budget=20, sinks=2, recent=3, nl=0x600000, kept=0x700000, N=3, **cache):
    c = _cache(**cache)
    return lib.sala_gla_kv_evict(ctypes.byref(c), budget, sinks, recent, _p(nl), _p(kept), N, None)


@no_gpu
@pytest.mark.parametrize("kw,want", CACHE_CASES)
def test_cache_argument_errors(lib, kw, want):
    assert _append(lib, **kw) == want
    assert _attend(lib, **kw) == want
    assert _evict(lib, **kw) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(N=1 << 19), INVALID), (dict(T=1 << 31), INVALID),
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(kld=255), INVALID), (dict(kld=260), INVALID),
    (dict(vld=0), INVALID), (dict(vld=1 << 33), INVALID), (dict(k=0x100008), MISALIGNED), (dict(v=0x200002), MISALIGNED),
    (dict(cu=0x3004), MISALIGNED), (dict(k=0x10000000 + 64), INVALID), (dict(v=0x30000000), INVALID),
    (dict(cu=0x20000008), INVALID), (dict(N=0), 0), (dict(N=0, table=0, lens=0), 0), (dict(T=0), 0),
    (dict(cu=0, N=1 << 17, T=1 << 15), INVALID), (dict(cu=0), CUDA), (dict(w=0), CUDA), (dict(kld=264), CUDA)])
def test_append_argument_errors(lib, kw, want):
    assert _append(lib, **kw) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(Hq=0), INVALID), (dict(Hq=33), INVALID), (dict(Hq=258), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=0), INVALID), (dict(o=0), INVALID), (dict(ld=4095), INVALID), (dict(ld=4100), INVALID),
    (dict(q=0x100004), MISALIGNED), (dict(o=0x400008), MISALIGNED), (dict(lse=0x500002), MISALIGNED),
    (dict(o=0x100000 + 64), INVALID), (dict(lse=0x400000 + 64), INVALID), (dict(lse=0x100000), INVALID),
    (dict(o=0x10000000), INVALID), (dict(lse=0x30000000), INVALID), (dict(o=0x1000), INVALID), (dict(lse=0x2000), INVALID),
    (dict(w=0), INVALID), (dict(w=0, acc=0), CUDA), (dict(lse=0), CUDA), (dict(N=0), 0), (dict(T=0), 0),
    (dict(Hq=256, ld=32768), CUDA), (dict(acc=0), CUDA), (dict(ld=4104), CUDA)])
def test_attention_argument_errors(lib, kw, want):
    assert _attend(lib, **kw) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(budget=0), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID), (dict(sinks=18), INVALID),
    (dict(sinks=21, recent=0), INVALID), (dict(budget=1 << 31), INVALID), (dict(w=0), INVALID), (dict(N=-1), INVALID),
    (dict(nl=0x600002), MISALIGNED), (dict(kept=0x700001), MISALIGNED), (dict(nl=0x2000), INVALID), (dict(kept=0x1000), INVALID),
    (dict(nl=0x700004), INVALID), (dict(kept=0x10000000), INVALID), (dict(N=0), 0), (dict(nl=0), CUDA), (dict(kept=0), CUDA),
    (dict(sinks=17), CUDA), (dict(), CUDA)])
def test_evict_argument_errors(lib, kw, want):
    assert _evict(lib, **kw) == want


def _logprobs(lib, x=0x100000, ld=1000, dt=0, tok=0x200000, lp=0x210000, ent=0x220000, ids=0x230000, vals=0x240000, N=2, V=1000,
              M=3, K=4):
    return lib.sala_gla_token_logprobs(_p(x), ld, dt, _p(tok), _p(lp), _p(ent), _p(ids), _p(vals), N, V, M, K, None)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), INVALID), (dict(V=0), INVALID), (dict(V=(1 << 20) + 1, ld=1 << 21), INVALID), (dict(M=-1), INVALID),
    (dict(K=-1), INVALID), (dict(K=65), INVALID), (dict(dt=2), INVALID), (dict(ld=999), INVALID), (dict(ld=1 << 33), INVALID),
    (dict(x=0), INVALID), (dict(tok=0), INVALID), (dict(lp=0), INVALID), (dict(ids=0), INVALID), (dict(vals=0), INVALID),
    (dict(x=0x100002), MISALIGNED), (dict(x=0x100001, dt=1), MISALIGNED), (dict(tok=0x200002), MISALIGNED),
    (dict(lp=0x210001), MISALIGNED), (dict(ent=0x220002), MISALIGNED), (dict(vals=0x240003), MISALIGNED),
    (dict(lp=0x100004), INVALID), (dict(ent=0x200004), INVALID), (dict(ids=0x210000), INVALID), (dict(vals=0x230008), INVALID),
    (dict(N=0), 0), (dict(M=0, K=0, ent=0, tok=0, lp=0, ids=0, vals=0), 0), (dict(x=0x100002, dt=1), CUDA), (dict(ent=0), CUDA),
    (dict(M=0, tok=0, lp=0), CUDA), (dict(K=0, ids=0, vals=0), CUDA), (dict(), CUDA)])
def test_logprobs_argument_errors(lib, kw, want):
    assert _logprobs(lib, **kw) == want
