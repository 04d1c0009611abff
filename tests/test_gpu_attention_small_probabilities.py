"""Probabilities far below a row's largest one: each is small, all together are not.

The tolerance of one output: its rounding; a probability's rounding, (2 D + 8) 2^-24 of the largest
sum of magnitudes behind a score (its exponent) and 2^-20 for the exponential; an fp32 sum over a
chunk's part of a wave and the joins; and 2^-40 of the row's largest for each probability, where it
falls below the type's normal numbers (fp16 holds 2^15 times it: 2^-25 / 2^15).
"""
import math

import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("n", [3000, 131001])
@pytest.mark.parametrize("bits", [13.0, 20.0, 23.6, 25.01, 27.0, 30.0])
def test_one_key_above_many(bits, n, kind):
    """One key with nearly all of the weight and a value of zero (a place that takes what attention
    is not wanted); what is left is the sum of thousands of probabilities 2^-bits of it."""
    D, page = 64, 64
    top = torch.tensor(bits * math.log(2), dtype=torch.float16)
    g = torch.Generator().manual_seed(n + int(bits))
    pages = -(-n // page)
    cache = torch.float8_e4m3fn if kind == "e4m3" else torch.float16
    k = torch.zeros((pages * page, D))
    v = torch.randint(8, 17, (pages * page, D), generator=g) / 8.0  # exact in either type
    place = n // 3
    k[place, 0], v[place] = 1.0, 0.0
    q = torch.zeros((1, 1, D), dtype=torch.float16)
    q[0, 0, 0] = top
    table = torch.arange(pages, dtype=torch.int32).view(1, pages)
    lengths = torch.tensor([n], dtype=torch.int32)
    caches = [t.view(pages, page, 1, D).to(cache).to(DEV) for t in (k, v)]
    lse = torch.full((1, 1), math.nan, dtype=torch.float32, device=DEV)
    out = tcm.paged_attention(q.to(DEV), *caches, table.to(DEV), lengths.to(DEV), scale=1.0, lse=lse)
    ref, rlse, mag, most = ol.paged_attention(q.double().numpy(), k.double().numpy().reshape(pages, page, 1, D),
                                              v.double().numpy().reshape(pages, page, 1, D), table.numpy(), [n], page, 1.0)
    ds = (2 * D + 8) * 2.0 ** -24 * most + 2.0 ** -20
    rel = 2.0 ** -12 + 2 * ds[..., None] + 400 * 2.0 ** -24
    err = np.abs(out.double().cpu().numpy() - ref)
    tol = rel * 2 * mag + 1.01 * ol.half_ulp(ref, "f16") + n * 2.0 ** -40 * 2.0
    assert (err <= tol).all(), f"worst {np.nanmax(err / tol)}: {out.flatten()[:3]} against {ref.flatten()[:3]}"
    assert abs(float(lse) - rlse[0, 0]) <= ds[0, 0] + 1e-5
