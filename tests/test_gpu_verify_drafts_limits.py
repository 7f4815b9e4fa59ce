"""The verification of drafted tokens at the ends of its range. What is expected is worked out by hand."""
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
