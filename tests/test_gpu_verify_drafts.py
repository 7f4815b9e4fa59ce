"""Verification of drafted tokens (sala_gla_verify_drafts) against the oracle. The results are whole
numbers and the sums behind them are exact, so every comparison is for equality."""
import pytest
import torch

from oracle import speculative as sp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_linear_attention_gb300 import build, sala_gla
    build.build()
    return sala_gla


def _case(N, K, V, dtype, drafter, ragged, seed, sharp=3.0):
    gen = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn(N, K + 1, V, generator=gen)
    d = (logits[:, :K] + 0.7 * torch.randn(N, K, V, generator=gen)).softmax(-1)
    x = torch.multinomial(d.reshape(N * K, V), 1, generator=gen).reshape(N, K).to(torch.int32) if K else \
        torch.zeros(N, 0, dtype=torch.int32)
    return dict(p=logits.softmax(-1).to(dtype), q=d.to(dtype) if drafter else None, x=x,
                u=torch.rand(N, K, generator=gen), s=torch.rand(N, generator=gen),
                counts=torch.randint(0, K + 1, (N,), generator=gen, dtype=torch.int32) if ragged else None)


def _gpu(t):
    return t.cuda() if t is not None else None


def _check(sg, c, status=0):
    tokens, accepted = sg.verify_drafts(_gpu(c["p"]), _gpu(c["q"]), _gpu(c["x"]), _gpu(c["u"]), _gpu(c["s"]),
                                        num_drafts=_gpu(c["counts"]))
    assert sg.get_device_status() == status
    t, a = sp.verify_drafts(c["p"], c["q"], c["x"], c["u"], c["s"], c["counts"])
    assert accepted.tolist() == a.tolist()
    assert tokens.tolist() == t.tolist()
    return t, a


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("N,K,V", [(1, 1, 1), (3, 2, 2), (2, 0, 97), (5, 3, 33), (7, 4, 1000), (1, 5, 50021),
                                   (33, 2, 4099), (2, 40, 511), (4, 1, 65536), (300, 1, 130)])
def test_small(sg, N, K, V, drafter, dtype):
    _check(sg, _case(N, K, V, dtype, drafter, N % 2 == 1, seed=N + K + V))


@pytest.mark.parametrize("V", [131072, 151337])
def test_large_vocabulary(sg, V):
    t, a = _check(sg, _case(6, 3, V, torch.float32, True, False, seed=9, sharp=1.0))


def test_largest_vocabulary(sg):
    _check(sg, _case(1, 1, 1 << 20, torch.bfloat16, False, False, seed=5, sharp=1.0))


def test_certain_and_impossible_drafts(sg):
    c = _case(4, 3, 500, torch.float32, True, False, seed=2)
    c["p"][:, :3], c["x"][:] = c["q"], c["q"].argmax(-1)     # equal distributions: always accepted
    assert _check(sg, c)[1].tolist() == [3] * 4
    c["p"][1, 1], c["p"][1, 1, (int(c["x"][1, 1]) + 1) % 500] = 0.0, 1.0   # the draft is impossible
    assert _check(sg, c)[1].tolist() == [3, 1, 3, 3]


@pytest.mark.parametrize("s", [0.0, 0.9999999403953552, 1.0, 7.0, -1.0, float("nan"), float("inf")])
def test_edges_of_the_draw(sg, s):
    c = _case(5, 2, 257, torch.float32, True, True, seed=4)
    c["s"][:] = s
    c["p"][0, :, :3] = 0.0
    c["p"][1, :, -5:] = 0.0
    _check(sg, c)


def test_rows_with_nothing_in_them(sg):
    c = _case(6, 2, 129, torch.float32, True, False, seed=6)
    c["p"][0] = 0.0                       # nothing anywhere: no token
    c["p"][1, 0] = float("nan")
    c["p"][2, 0] = -1.0
    c["p"][3, 0], c["q"][3, 0], c["u"][3] = 0.25, 0.25, 1.0   # all of it is the drafter's: the target
    c["p"][4, 0], c["q"][4, 0] = float("inf"), 0.0            # counts as one each
    c["u"][5] = float("nan")                                  # never accepted
    t, a = _check(sg, c)
    assert t[:3, 0].tolist() == [-1] * 3 and a[3] == 0 and t[3, 0] >= 0


def test_tokens_and_counts_outside_their_range(sg):
    c = _case(6, 4, 300, torch.float32, True, False, seed=8)
    c["x"][2, 1] = -1                                # the row's drafts end: not an error
    _check(sg, c)
    c["x"][4, 0] = 300                               # past the vocabulary: reported
    _check(sg, c, status=8)
    c["x"][4, 0], c["counts"] = 3, torch.tensor([4, 5, 0, -2, 1, 4], dtype=torch.int32)
    _check(sg, c, status=8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_padded_vocabulary_and_odd_rows(sg, dtype):
    # rows longer than the vocabulary, and rows whose starts are not aligned alike in p and q
    c = _case(9, 3, 1021, dtype, True, False, seed=12)
    want = sp.verify_drafts(c["p"], c["q"], c["x"], c["u"], c["s"])
    for p_ld, q_ld, shift in ((1024, 1024, 0), (1021, 1027, 1), (1030, 1021, 3)):
        P = torch.full((9 * 4 * p_ld + 8,), 0.5, dtype=dtype, device="cuda")
        Q = torch.zeros(9 * 3 * q_ld + 8, dtype=dtype, device="cuda")
        p = P[shift:shift + 36 * p_ld].view(9, 4, p_ld)[:, :, :1021]
        q = Q[:27 * q_ld].view(9, 3, q_ld)[:, :, :1021]
        p.copy_(c["p"])
        q.copy_(c["q"])
        tokens, accepted = sg.verify_drafts(p, q, c["x"].cuda(), c["u"].cuda(), c["s"].cuda())
        assert tokens.tolist() == want[0].tolist() and accepted.tolist() == want[1].tolist()
    with pytest.raises(ValueError):
        sg.verify_drafts(p.transpose(0, 1).contiguous().transpose(0, 1), q, c["x"].cuda(), c["u"].cuda(),
                         c["s"].cuda())
    assert sg.get_device_status() == 0


def test_graph_and_side_stream(sg):
    c = _case(8, 3, 5000, torch.float32, True, False, seed=21)
    d = {n: _gpu(c[n]) for n in ("p", "q", "x", "u", "s")}
    tokens, accepted = torch.empty(8, 4, dtype=torch.int32, device="cuda"), torch.empty(8, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = sp.verify_drafts(c["p"], c["q"], c["x"], c["u"], c["s"])
    t, a = sg.verify_drafts(d["p"], d["q"], d["x"], d["u"], d["s"], stream=side)
    side.synchronize()
    assert t.tolist() == want[0].tolist() and a.tolist() == want[1].tolist()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.verify_drafts(d["p"], d["q"], d["x"], d["u"], d["s"], tokens=tokens, accepted=accepted)
    c2 = _case(8, 3, 5000, torch.float32, True, False, seed=22)
    for n in d:
        d[n].copy_(c2[n])
    graph.replay()
    want = sp.verify_drafts(c2["p"], c2["q"], c2["x"], c2["u"], c2["s"])
    assert tokens.tolist() == want[0].tolist() and accepted.tolist() == want[1].tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V", [(3, 3000), (3, 17001), (3, 40008), (3, 70001), (700, 20000), (400, 60001)])
@pytest.mark.parametrize("drafter", [True, False])
def test_values_of_every_kind(sg, N, V, dtype, drafter):
    # probabilities that are none, borders between two units, and rows cut into one to eight parts of a cluster
    c = _case(N, 1, V, dtype, drafter, False, seed=N + V, sharp=6.0)
    gen = torch.Generator().manual_seed(V)
    for t in (c["p"], c["q"]) if drafter else (c["p"],):
        flat = t.view(N, -1)
        for value in (float("nan"), float("inf"), -1.0, -0.0, 2.0 ** -44, 3 * 2.0 ** -44, 5 * 2.0 ** -44, 2.0 ** -130):
            flat.scatter_(1, torch.randint(0, flat.shape[1], (N, 6), generator=gen), value)
        flat[:, 7] = 1.5
    _check(sg, c)
