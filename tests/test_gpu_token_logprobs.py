"""Log probabilities, entropy and top alternatives against the plain form in 64 bits.

Bounds: with x the logits and m their maximum, x - m is one rounded subtraction (relative 2^-24), exp is
good to 2 units (2^-22), and sums of n positive terms over threads are off by at most the length of a thread's own
chain, V / 256 here, plus the tree, times 2^-24. So lse - m is off by at most (V / 256 + 40) 2^-24, and a log
probability by that, the rounding of x - m and its own: |lp| 2^-22. The entropy's second sum has terms e^d |d|
<= 1 / e each relative to the same error plus 2^-22 from e, and one more division: it is off by at most
(V / 256 + 60) 2^-24 (1 + |entropy| + log V)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _check(x, tokens, top, entropy=True, view=None):
    from gated_linear_attention_gb300 import sala_gla
    from oracle import softmax_layers as ref
    d = x.cuda() if view is None else view
    got = sala_gla.token_logprobs(d, None if tokens is None else tokens.cuda(), top=top, entropy=entropy)
    lp, ent, ids, vals = ref.logprobs(x, tokens, top)
    V = x.shape[1]
    tol = (V / 256 + 40) * 2.0 ** -24
    def near(a, b):
        a, b = a.cpu().double(), b.double()
        fin = b.isfinite()
        assert torch.equal(a[~fin], b[~fin])
        assert bool(((a - b)[fin].abs() <= tol + b[fin].abs() * 2.0 ** -22).all()), float((a - b)[fin].abs().max())
    if tokens is not None:
        near(got[0], lp)
    if entropy:
        e = got[1].cpu().double()
        assert bool(((e - ent).abs() <= (V / 256 + 60) * 2.0 ** -24 * (1 + ent.abs() + math.log(V))).all())
    else:
        assert got[1] is None
    if top:
        assert torch.equal(got[2].cpu(), ids)
        near(got[3], vals)
    else:
        assert got[2] is None and got[3] is None
    return sala_gla.get_device_status()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,M,top", [(1, 1, 1, 1), (1, 7, 2, 10), (3, 33, 1, 5), (2, 1000, 3, 64), (5, 4099, 1, 20),
                                       (2, 16384, 1, 1), (1, 50021, 2, 32), (1, 65537, 1, 0), (37, 129, 4, 8)])
def test_logprobs(dtype, N, V, M, top):
    gen = torch.Generator().manual_seed(V)
    x = (3 * torch.randn(N, V, generator=gen)).to(dtype)
    tokens = torch.randint(0, V, (N, M), generator=gen, dtype=torch.int32)
    assert _check(x, tokens, top) == 0


def test_one_token_a_row_and_nothing_asked():
    from gated_linear_attention_gb300 import sala_gla
    x = torch.randn(4, 100)
    assert _check(x, torch.tensor([3, 99, 0, -1], dtype=torch.int32), 0, entropy=False) == 0
    assert _check(x, None, 3) == 0
    assert sala_gla.token_logprobs(x.cuda(), entropy=False) == (None, None, None, None)
    out = sala_gla.token_logprobs(x[:0].cuda(), torch.zeros(0, 2, dtype=torch.int32, device="cuda"), top=2)
    assert [tuple(t.shape) for t in out] == [(0, 2), (0,), (0, 2), (0, 2)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 3001, 70001])
def test_ties_and_values_of_every_kind(dtype, V):
    """Equal logits go to the lower token, however many there are; NaN, infinities, masked vocabularies."""
    gen = torch.Generator().manual_seed(V)
    x = torch.zeros(9, V)
    x[1] = torch.randint(0, 3, (V,), generator=gen).float()
    x[2] = -math.inf
    x[2, [3, 17]] = torch.tensor([-2.0, 1.0])
    x[3] = -math.inf
    x[4] = torch.randn(V, generator=gen)
    x[4, [2, 30]] = math.nan
    x[5] = torch.randn(V, generator=gen)
    x[5, [5, 35]] = math.inf
    x[6] = math.nan
    x[7] = torch.linspace(-50, 50, V)
    x[8] = torch.finfo(dtype).min          # the type's lowest value as a mask
    x[8, 11] = 0.5
    tokens = torch.tensor([[0, 5, 39, 17]] * 9, dtype=torch.int32)
    assert _check(x.to(dtype), tokens, 16) == 0


def test_zeros_of_both_signs_are_equal():
    from gated_linear_attention_gb300 import sala_gla
    x = torch.full((1, 600), -1.0)
    x[0, [5, 300]] = -0.0
    x[0, [9, 401]] = 0.0
    assert sala_gla.token_logprobs(x.cuda(), top=4)[2].tolist() == [[5, 9, 300, 401]]


def test_large_vocabulary_and_overflowing_ties():
    x = torch.zeros(2, 1 << 20)
    x[1, 1 << 19:] = 1.0
    x[1, (1 << 20) - 1] = 2.0
    from gated_linear_attention_gb300 import sala_gla
    lp, ent, ids, vals = sala_gla.token_logprobs(x.cuda(), torch.tensor([[7], [7]], dtype=torch.int32).cuda(), top=3)
    assert ids.tolist() == [[0, 1, 2], [(1 << 20) - 1, 1 << 19, (1 << 19) + 1]]
    want = x.double().log_softmax(1)
    assert float((lp.cpu().double()[:, 0] - want[:, 7]).abs().max()) <= (4096 + 40) * 2.0 ** -24
    assert float((ent.cpu().double() + (want.exp() * want).sum(1)).abs().max()) <= (4096 + 60) * 2.0 ** -24 * 30


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off,pad", [(0, 3), (1, 0), (1, 5), (3, 8)])
def test_rows_apart_and_off_alignment(dtype, off, pad):
    gen = torch.Generator().manual_seed(off + pad)
    V = 2003
    buf = torch.full((4 * (V + pad) + off,), 50.0, dtype=dtype)
    rows = buf[off:].reshape(4, V + pad)[:, :V]
    rows.copy_(torch.randn(4, V, generator=gen))
    dev = buf.cuda()[off:].reshape(4, V + pad)[:, :V]
    assert _check(rows, torch.tensor([[1], [2], [2002], [0]], dtype=torch.int32), 7, view=dev) == 0


def test_tokens_out_of_range():
    x = torch.randn(3, 50)
    assert _check(x, torch.tensor([[50], [3], [-5]], dtype=torch.int32), 2) == 8
    assert _check(x, torch.tensor([[2 ** 31 - 1], [-2 ** 31], [1]], dtype=torch.int32), 0) == 8


def test_streams_graphs_and_repeats():
    from gated_linear_attention_gb300 import sala_gla
    x, t = torch.randn(33, 30011, device="cuda"), torch.zeros(33, 1, dtype=torch.int32, device="cuda")
    want = sala_gla.token_logprobs(x, t, top=9)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    other = sala_gla.token_logprobs(x, t, top=9, stream=s)
    s.synchronize()
    with torch.cuda.graph(graph):
        third = sala_gla.token_logprobs(x, t, top=9)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals():
    from gated_linear_attention_gb300 import sala_gla
    x, t = torch.randn(3, 50, device="cuda"), torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    for call, err in ((lambda: sala_gla.token_logprobs(x.half(), t), TypeError),
                      (lambda: sala_gla.token_logprobs(x.cpu(), t), ValueError),
                      (lambda: sala_gla.token_logprobs(x, t.long()), TypeError),
                      (lambda: sala_gla.token_logprobs(x, t[:2]), ValueError),
                      (lambda: sala_gla.token_logprobs(x.t(), t), ValueError),
                      (lambda: sala_gla.token_logprobs(x, t, top=65), sala_gla.SalaError),
                      (lambda: sala_gla.token_logprobs(x, t, top=-1), sala_gla.SalaError)):
        with pytest.raises(err):
            call()
