"""Every bf16 value into an e4m3 cache, at scales over the whole range: the byte of the rounded quotient, its sign too."""
import pytest
import torch

from paged_inputs import bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scales", [(1e-12, 1e12), (3.1e-5, 0.0173), (1.0, 7.3), (2.0 ** -9, 448.0), (0.1, 1 / 3)])
def test_every_value(scales):
    from gated_linear_attention_gb300 import sala_gla
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)    # all bit patterns
    T = (1 << 16) // 128
    k = x.reshape(T, 1, 128).expand(T, 2, 128).contiguous()
    scale = torch.tensor(scales, dtype=torch.float32)
    pages = [torch.zeros(T // 16, 2, 16, 128, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    cache = sala_gla.KvCache(*pages, torch.arange(T // 16, dtype=torch.int32, device="cuda")[None],
                             torch.tensor([T], dtype=torch.int32, device="cuda"), scale.cuda(), scale.flip(0).contiguous().cuda())
    sala_gla.kv_append(cache, k.cuda()[None], k.cuda()[None])
    assert sala_gla.get_device_status() == 0
    for got, by in ((pages[0], scale), (pages[1], scale.flip(0))):
        want = (k.float() / by[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        got = got.cpu().transpose(1, 2).reshape(T, 2, 128)
        nan = k.isnan()
        assert torch.equal(got.float().isnan(), nan)
        assert torch.equal(bits(got)[~nan], bits(want)[~nan])
