"""The codes that append writes into an E4M3 cache, to the bit."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, FH, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def test_codes_to_the_bit(K):
    """Every half-precision value but NaN against several scales: the very codes of the quotients, zeros' signs among them."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    for dtype in (BF, FH):
        x = every.view(dtype).view(64, 1, 16, 64).cuda()
        scales = torch.tensor([1.0, 0.3, 1e-3, 7.1, 448.0, 3e-20, 1e20, 1.0000001, 0.9999999, 0.017, 2.0 ** -130, 3.0, 0.1, 65504.0, 1e-8, 5e-4])
        cache = K.KdaKvCache.zeros(1, 64, 16, 64, 1, 16, 64, dtype=E4, k_scale=scales.view(1, 16).cuda(), v_scale=scales.flip(0).view(1, 16).cuda())
        rows = torch.arange(64, dtype=torch.int32, device="cuda")
        K.kda_kv_extend(cache, rows, 1)
        K.kda_kv_append(cache, 0, rows, x, x)
        for got, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            got = got[0, :, :, 0].view(torch.uint8)
            want = (x[:, 0].float() / s.view(1, 16, 1)).clamp(-448, 448).to(E4).view(torch.uint8)
            nan = x[:, 0].isnan()
            assert torch.equal(got[~nan], want[~nan])
            assert ((got[nan] & 0x7f) == 0x7f).all()
