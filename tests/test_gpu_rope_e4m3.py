"""E4M3 caches hold the code of x / scale for every scale, to the last bit."""
import pytest
import torch

import tensor_core_matrix_amd as tcm

pytestmark = pytest.mark.gpu
DEV = "cuda"


def every_half(dt):
    """Every 16-bit number as (1024, 1, 64)."""
    return torch.arange(-2**15, 2**15, dtype=torch.int32).to(torch.int16).view(dt).view(-1, 1, 64)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("scale", [0.640625, 0.03, 0.1, 1 / 3, 0.0125, 7.7, 448.0, 1e-30, 1e30, 1e-39, 2.0 ** -126])
def test_e4m3_codes_are_of_the_quotient(scale, dt):
    """Keys (not normed, not rotated) and values: the E4M3 code of the fp32 quotient, for every
    number of the type, ties among them."""
    x = every_half(dt)
    T = x.shape[0]
    s = torch.tensor(scale, dtype=torch.float32)
    want = (x.float() / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    kc = torch.zeros((T, 1, 1, 64), dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    xd = x.to(DEV)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    tcm.qk_norm_rope_cache(xd, xd, xd, None, None, kc, vc, slots, norm=False, k_scale=float(s), v_scale=float(s))
    for c in (kc, vc):
        got = c.view(torch.float8_e4m3fn).float().cpu().view(want.shape)
        same = (got == want) | (torch.isnan(got) & torch.isnan(want))
        assert same.all(), (int((~same).sum()), x[~same][:4], got[~same][:4], want[~same][:4])
