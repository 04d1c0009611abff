"""Infinite elements of an adapter's B times finite inner products: infinities of their sign in the
adapter's rows, in any number of rows."""
import math

import pytest
import torch

import tensor_core_matrix_amd as tcm
from test_gpu_lora_range import SIZES, adapters

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dt,odt", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16),
                                    (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("how", ["one", "two", "many"])
@pytest.mark.parametrize("M,N", SIZES)
def test_infinite_b(M, N, how, dt, odt):
    """Column 3 of every adapter +infinity at rank 2, column 7 -infinity; t there is every size of two
    magnitudes, numbers that one part holds among them."""
    K, R, L = 8, 8, 5
    g = torch.Generator().manual_seed(M)
    x = torch.zeros((M, K))
    x[:, 0] = torch.randint(1, 500, (M,), generator=g) / 128.0
    x[::3, 0], x[1::3, 0] = 1.0, -0.5
    x = x.to(dt).to(DEV)
    a = torch.zeros((L, R, K), dtype=dt, device=DEV)
    a[:, :, 0] = 1.0
    b = torch.ones((L, N, R), dtype=dt, device=DEV)
    b[:, 3, 2], b[:, 7, 2] = math.inf, -math.inf
    w = torch.zeros((N, K), dtype=dt, device=DEV)
    rows = adapters(M, how)
    out = tcm.lora_gemm_tn(x, w, a, b, rows, out_dtype=odt)
    t = x[:, 0].float()
    want = (8 * t).to(odt)[:, None].repeat(1, N)
    want[:, 3], want[:, 7] = torch.sign(t) * math.inf, -torch.sign(t) * math.inf
    want[rows < 0] = 0
    assert torch.equal(out, want)
