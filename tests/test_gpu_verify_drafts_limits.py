"""The verification of drafted tokens at the ends of its range: the largest sum that a row can have, and
values that are no probabilities in the accept test. What is expected is worked out by hand."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_linear_attention_gb300 import build, sala_gla
    build.build()
    return sala_gla


def _call(sg, p, q, x, u, s):
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda t: torch.tensor(t, dtype=torch.float32, device="cuda")  # noqa: E731
    tokens, accepted = sg.verify_drafts(p, q, i32(x), f32(u), f32(s), tokens=torch.full((len(s), p.shape[1]), -7, dtype=torch.int32, device="cuda"))
    assert sg.get_device_status() == 0
    return tokens.tolist(), accepted.tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_largest_sum(sg, dtype):
    # 2^20 values that count as 1 each, 2^43 units: 2^63 in all. Token = the whole part of s 2^20.
    V = 1 << 20
    s = [0.0, 0.25, 0.5, 0.75, 1.0 - 2.0 ** -24]
    want = [int(x * V) for x in s]
    p = torch.full((5, 1, V), 1.0, dtype=dtype, device="cuda")
    p[1::2] = 3.0
    none = [[]] * 5
    assert _call(sg, p, None, none, none, s) == ([[t] for t in want], [0] * 5)
    p = torch.ones(5, 2, V, dtype=dtype, device="cuda")
    x = [[7]] * 5
    # a rejected draft of a drafter that gave every token nothing: the same sum
    assert _call(sg, p, torch.zeros(5, 1, V, dtype=dtype, device="cuda"), x, [[float("nan")]] * 5, s) == \
        ([[t, -1] for t in want], [0] * 5)
    # ... that gave it all: nothing is left, the draw is from the target
    assert _call(sg, p, torch.ones(5, 1, V, dtype=dtype, device="cuda"), x, [[1.0]] * 5, s) == ([[t, -1] for t in want], [0] * 5)
    # ... without probabilities: one token less
    t, a = _call(sg, p, None, x, [[1.0]] * 5, s)
    assert a == [0] * 5 and t == [[int(x * (V - 1)) + (int(x * (V - 1)) >= 7), -1] for x in s]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_accept_test_takes_values_as_probabilities(sg, dtype):
    # (p(x), q(x), u) of a drafted token: below 0 and NaN count as 0, above 1 as 1
    nan, inf = float("nan"), float("inf")
    rows = [(0.0, -1.0, 0.5, False), (0.5, -1.0, 0.5, True), (0.25, nan, 0.5, True), (0.0, nan, 0.5, False), (nan, 0.5, 0.0, False),
            (-1.0, 0.5, 0.0, False), (-1.0, -4.0, 0.5, False), (0.75, 2.0, 0.5, True), (0.75, inf, 0.5, True),
            (2.0, 1.5, 1.0, False), (inf, 1.0, 1.0, False), (inf, inf, 0.5, True), (0.75, 1.0, 0.75, False), (0.5, 0.5, 0.5, True)]
    N = len(rows)
    p, q = torch.zeros(N, 2, 40, dtype=dtype), torch.zeros(N, 1, 40, dtype=dtype)
    p[:, :, 3], q[:, :, 30] = 1.0, 1.0
    for n, (a, b, _, _) in enumerate(rows):
        p[n, 0, 9], q[n, 0, 9] = a, b
    _, accepted = _call(sg, p.cuda(), q.cuda(), [[9]] * N, [[r[2]] for r in rows], [0.0] * N)
    assert accepted == [int(r[3]) for r in rows]
