"""The adapters' inner product t over the whole range of its type: more than 64 rows multiply it in
16-bit parts, which must neither overflow nor run out of digits.

Tolerance: fp32 sums of n terms are off by at most n 2^-24 of the sum of magnitudes; the two fp16
parts of t hold 22 bits of the largest of 16 ranks, which is 2^-22 of a sum over ranks at most 16
times that of one: 2^-18 of the sum of magnitudes; fp32 outputs of bf16 hold t whole.
"""
import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol

pytestmark = pytest.mark.gpu
DEV = "cuda"

# rows and columns that take each of the tiles (64 x 64, 128 x 64, 128 x 128, 256 x 256 with 256 compute
# units), and the row kernel beside them
SIZES = [(64, 100), (65, 100), (128, 12225), (128, 32641), (256, 65281)]


def f64(t):
    return t.double().cpu().numpy()


def adapters(M, how):
    """All of one adapter; two a block of 16; one a row."""
    i = torch.arange(M)
    rows = {"one": 0 * i, "two": (i // 8) % 3 - 1, "many": i % 6 - 1}[how]
    return rows.to(torch.int32).to(DEV)


@pytest.mark.parametrize("how", ["one", "two", "many"])
@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("tx,bx", [(2.0 ** 20, 2.0 ** -12), (2.0 ** -12, 2.0 ** 8), (2.0 ** -24, 2.0 ** 12)])
def test_f16_inner_products_of_any_size(tx, bx, M, N, how):
    """t of about `tx` by way of the scale; columns that are bits of one sign or the other."""
    K, R, L = 16, 24, 5
    g = torch.Generator().manual_seed(M)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, a = n(M, K).half().to(DEV), n(L, R, K).half().to(DEV)
    b = (n(L, N, R) * bx).half().to(DEV)
    w = torch.zeros((N, K), dtype=torch.float16, device=DEV)
    scales = (tx * (0.5 + torch.rand((L,), generator=g))).to(DEV)
    rows = adapters(M, how)
    at = np.unique(np.linspace(0, N - 1, 150).astype(int))
    out = tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales, out_dtype=torch.float32)
    pick = torch.from_numpy(at).to(DEV)
    ref, s = ol.lora(f64(x), f64(w[pick]), f64(a), f64(b[:, pick]), rows.tolist(), f64(scales))
    err = np.abs(f64(out[:, pick]) - ref)
    tol = s * ((K + R + 16) * 2.0 ** -24 + 2.0 ** -18)
    assert (err <= tol).all(), f"worst {np.nanmax(err / np.maximum(tol, 1e-300))}"


@pytest.mark.parametrize("how", ["one", "two", "many"])
@pytest.mark.parametrize("M,N", SIZES)
def test_f32_outputs_of_bf16_hold_every_bit_of_t(M, N, how):
    """t = 1 + 2^-9 + 2^-17 has one bit in each of its three parts; sums of it are exact."""
    K, R, L = 8, 8, 5
    bf = torch.bfloat16
    x = torch.tensor([1.0, 2.0 ** -9, 2.0 ** -17, 0, 0, 0, 0, 0], device=DEV).to(bf).repeat(M, 1)
    a = torch.ones((L, R, K), dtype=bf, device=DEV)
    b = torch.ones((L, N, R), dtype=bf, device=DEV)
    b[:, 1::2] = -0.5
    w = torch.zeros((N, K), dtype=bf, device=DEV)
    rows = adapters(M, how)
    out = tcm.lora_gemm_tn(x, w, a, b, rows, out_dtype=torch.float32)
    want = torch.full((M, N), 8 * (1 + 2.0 ** -9 + 2.0 ** -17), device=DEV)
    want[:, 1::2] *= -0.5
    want[rows < 0] = 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M", [40, 100])
def test_infinite_and_largest_inner_products(M, dt):
    """An infinite t gives an infinite output; the largest finite fp32 values a finite one."""
    K, R, N = 8, 8, 48
    x = torch.ones((M, K), dtype=dt, device=DEV)
    a = torch.zeros((3, R, K), dtype=dt, device=DEV)
    a[:, 0, 0] = 1.0
    b = torch.zeros((3, N, R), dtype=dt, device=DEV)
    b[:, :, 0] = 2.0 ** -14
    w = torch.zeros((N, K), dtype=dt, device=DEV)
    big = 3.4028234e38
    scales = torch.tensor([float("inf"), big, -big], device=DEV)
    rows = (torch.arange(M) % 4 - 1).to(torch.int32).to(DEV)
    ranks = torch.ones(3, dtype=torch.int32, device=DEV)  # (an infinite factor of a zero is NaN)
    out = tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales, ranks=ranks, out_dtype=torch.float32)
    want = torch.tensor([0.0, float("inf"), big * 2.0 ** -14, -big * 2.0 ** -14], device=DEV)[rows.long() + 1]
    err = (out - want[:, None]).abs() / want.abs().clamp(min=1.0)[:, None]
    assert torch.equal(torch.isinf(out), torch.isinf(want)[:, None].expand(M, N))
    assert (err[torch.isfinite(out)] <= 2.0 ** -20).all()
