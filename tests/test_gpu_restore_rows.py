"""Every e4m3 code at every e8m0 scale: fp32 holds code * scale wherever it is
below 2^128; bf16 for scale bytes 3 to 246, rounded to nearest even below them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    from combine_route_mask_amd import ffn, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    return ffn


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_code_at_every_scale(F, dtype):
    codes = torch.arange(256, dtype=torch.uint8).view(8, 32).repeat(256, 1).view(torch.float8_e4m3fn)
    byte = torch.arange(256, dtype=torch.uint8).repeat_interleave(8).view(-1, 1)
    got = F.restore_rows(codes.cuda(), byte.view(torch.float8_e8m0fnu).cuda(), dtype=dtype).cpu().double()
    want = codes.float().double() * torch.exp2(byte.double() - 127)
    want[byte[:, 0] == 255] = float("nan")
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan)
    b = byte.expand(-1, 32).long()
    inside = ~nan & (want.abs() < 2.0 ** 128)
    exact = inside & ((b >= 3) & (b <= 246) if dtype == torch.bfloat16 else b >= 0)
    assert torch.equal(got[exact], want[exact])
    # fp32 holds all of these products: to bf16 there is one rounding, of numbers past its largest to infinity
    assert torch.equal(got[~nan], want[~nan].float().to(dtype).double())
