"""Padding rows of the decode step over drafted tokens: nothing that stands beside a negative slot is
read as an error. A batch padded to a captured size leaves old counts there."""
import pytest
import torch

from gated_linear_attention_gb300 import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_linear_attention_gb300 import build, sala_gla
    build.build()
    return sala_gla


@pytest.mark.parametrize("storage", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Tp", [(3, 4), (12, 16), (20, 2), (3, 40)])
@pytest.mark.parametrize("accepted,count", [(1 << 20, 0), (0, -5), (2 ** 31 - 1, 1 << 30), (-7, 41)])
def test_counts_of_a_padding_row_are_not_looked_at(sg, T, Tp, accepted, count, storage):
    gen = torch.Generator().manual_seed(T)
    q, k, pk = (inputs.l2_normalise(torch.randn(3, n, 2, 128, generator=gen)).to(torch.bfloat16).cuda() for n in (T, T, Tp))
    v, pv = (torch.randn(3, n, 2, 128, generator=gen).to(torch.bfloat16).cuda() for n in (T, Tp))
    g, pg = (-torch.rand(3, n, 2, generator=gen).cuda() for n in (T, Tp))
    pool = torch.randn(4, 2, 128, 128, generator=gen).to(storage).cuda()
    slots = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    outs = []
    for a, c in ((0, 1), (accepted, count)):
        d = pool.clone()
        o = sg.recurrent_draft_step(q, k, v, g, 0.125, d, slots, pending=(pk, pv, pg),
                                    accepted=torch.tensor([1, a, -1], dtype=torch.int32, device="cuda"),
                                    num_tokens=torch.tensor([T, c, 2], dtype=torch.int32, device="cuda"))
        assert sg.get_device_status() == 0
        outs.append((o, d))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.all(outs[1][0][1] == 0)
