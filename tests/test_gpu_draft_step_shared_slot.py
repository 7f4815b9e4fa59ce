"""Rows of the decode step over drafted tokens that commit nothing may share a slot (continuations of one
cached prefix): each gives what it gives alone, bit for bit, and the pool stays as it is."""
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


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Tp", [(4, 0), (4, 3), (16, 16), (19, 2)])
def test_rows_that_only_read_share_a_slot(sg, T, Tp, storage):
    N, H = 24, 8
    gen = torch.Generator(device="cuda").manual_seed(T + Tp)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    tok = [(0.1 * rand(N, T, H, 128)).to(torch.bfloat16) for _ in range(3)] + [-rand(N, T, H).abs()]
    pend = [(0.1 * rand(N, Tp, H, 128)).to(torch.bfloat16) for _ in range(2)] + [-rand(N, Tp, H).abs()] if Tp else None
    before = rand(3, H, 128, 128).to(storage)
    slots = torch.ones(N, dtype=torch.int32, device="cuda")
    none = torch.full((N,), -1, dtype=torch.int32, device="cuda") if Tp else None

    def call(rows):
        pool = before.clone()
        o = sg.recurrent_draft_step(*(t[rows] for t in tok), 0.125, pool, slots[rows],
                                    pending=tuple(t[rows] for t in pend) if Tp else None, accepted=none[rows] if Tp else None)
        assert sg.get_device_status() == 0 and torch.equal(pool, before)
        return o
    assert torch.equal(call(slice(0, N)), torch.cat([call(slice(n, n + 1)) for n in range(N)]))
