"""The e4m3 code of every 16-bit value, bit for bit the float32 division's, signs of zeros included."""
import pytest
import torch

import weight_only_int4_w4a16_amd as w

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_codes_of_every_value(dtype):
    every = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int16).view(dtype).view(512, 1, 128)
    scales = torch.tensor([1.0, 0.5, 0.0123, 3.0, 0.007, 1e-3, 448.0, 1.7e30, 2e-30, 1e-20, 2.0 ** -61, 1.1])
    heads = len(scales)
    x = every.expand(-1, heads, -1).contiguous()
    cache = torch.full((32, 16, heads, 128), 1.0).to(torch.float8_e4m3fn).cuda()
    other = cache.clone()
    slots = torch.arange(512, dtype=torch.int32, device="cuda")
    w.paged_kv_write(x.cuda(), x.cuda(), cache, other, slots, k_scale=scales.cuda(), v_scale=scales.flip(0).cuda())
    for got, s in ((cache, scales), (other, scales.flip(0))):
        want = (x.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        a, b = got.cpu().view(512, heads, 128).view(torch.uint8), want.view(torch.uint8)
        nan = want.float().isnan()
        assert torch.equal(a[~nan], b[~nan])
        assert bool(((a[nan] & 0x7F) == 0x7F).all())   # any NaN code will do
