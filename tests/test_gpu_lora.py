"""lora_gemm_tn on the GPU against the float64 oracle.

Tolerance: fp32 sums of n terms in any order are off by at most n 2^-24 of the sum of
magnitudes s; the adapter's inner product enters as two 16-bit values, off by 2^-16
(bf16) of its magnitude; the output is rounded once, half an ulp of its type.
"""
import math

import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float32: "f32"}


def f64(t):
    return t.double().cpu().numpy()


def draw(M, N, K, L, R, dt, seed, ldx=None):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g).to(dt).to(DEV)  # noqa: E731
    x = n(M, ldx or K)[:, :K]
    rows = torch.randint(-1, L, (M,), generator=g).to(torch.int32).to(DEV)
    scales = (0.5 + torch.rand((L,), generator=g)).to(DEV)
    return x, n(N, K), n(L, R, K), n(L, N, R), rows, scales


def check(out, x, w, a, b, rows, scales=None, ranks=None):
    ref, s = ol.lora(f64(x), f64(w), f64(a), f64(b), rows.tolist(),
                     None if scales is None else f64(scales), None if ranks is None else ranks.tolist())
    K, R = x.shape[1], a.shape[1]
    tol = s * ((K + R + 16) * 2.0 ** -24 + 2.0 ** -16) + ol.half_ulp(ref, NAMES[out.dtype]) * 1.01
    err = np.abs(f64(out) - ref)
    assert (err <= tol).all(), f"worst {np.nanmax(err / tol)} at {np.argwhere(~(err <= tol))[:4]}"


SIZES = [  # M, N, K, L, R
    (1, 16, 32, 1, 8), (1, 4096, 512, 3, 16), (2, 40, 8, 2, 8), (5, 100, 1000, 4, 16), (16, 33, 264, 5, 24),
    (17, 50, 520, 40, 32), (31, 64, 2048, 3, 64), (48, 96, 328, 64, 16), (64, 130, 96, 7, 128),
    (65, 70, 200, 5, 8), (100, 257, 72, 100, 16), (128, 128, 64, 2, 16), (200, 300, 136, 6, 40),
    (257, 129, 640, 9, 16),
]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(size, dt):
    x, w, a, b, rows, scales = draw(*size, dt, 100 + size[0])
    for odt in (dt, torch.float32):
        out = torch.full((size[0], size[1]), math.nan, dtype=odt, device=DEV)
        assert tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales, out=out) is out
        check(out, x, w, a, b, rows, scales)


@pytest.mark.parametrize("M", [3, 40, 70, 600])
def test_runs_of_rows(M):
    """Requests of consecutive rows whose ends fall inside blocks and tiles, some without
    an adapter; no scales."""
    x, w, a, b, _, _ = draw(M, 136, 256, 4, 16, torch.bfloat16, 7)
    rows = torch.tensor([(i * 7 // M) % 5 - 1 for i in range(M)], dtype=torch.int32, device=DEV)
    check(tcm.lora_gemm_tn(x, w, a, b, rows), x, w, a, b, rows)


@pytest.mark.parametrize("M,N", [(2048, 2056), (1100, 4100)])
def test_many_tiles(M, N):
    """The larger tiles: every adapter path at the edges of both dimensions."""
    x, w, a, b, rows, scales = draw(M, N, 136, 6, 16, torch.bfloat16, 8)
    check(tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales), x, w, a, b, rows, scales)


@pytest.mark.parametrize("M", [5, 40, 150])
def test_strided_rows(M):
    """x a slice of wider rows, out a slice of a wider tensor (odd row length: element
    stores), whose other elements stay."""
    x, w, a, b, rows, scales = draw(M, 52, 200, 3, 16, torch.float16, 9, ldx=256)
    wide = torch.full((M, 61), 7.0, dtype=torch.float16, device=DEV)
    out = wide[:, :52]
    tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales, out=out)
    check(out, x, w, a, b, rows, scales)
    assert (wide[:, 52:] == 7.0).all()


@pytest.mark.parametrize("M", [1, 20, 90])
def test_ranks_hide_what_lies_beyond(M):
    """Rows of A and columns of B past an adapter's rank hold NaN; ranks are clipped."""
    L, R = 6, 32
    x, w, a, b, _, scales = draw(M, 48, 64, L, R, torch.bfloat16, 10)
    ranks = [32, 8, 0, 13, 99, -4]
    for l, r in enumerate(ranks):
        r = min(max(r, 0), R)
        a[l, r:] = math.nan
        b[l, :, r:] = math.nan
    rows = torch.tensor([i % (L + 1) - 1 for i in range(M)], dtype=torch.int32, device=DEV)
    ranks = torch.tensor(ranks, dtype=torch.int32, device=DEV)
    out = tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales, ranks=ranks)
    check(out, x, w, a, b, rows, scales, ranks)


@pytest.mark.parametrize("M", [4, 40, 200])
def test_one_bad_adapter_stays_with_its_rows(M):
    """Infinities and NaN in adapter 1 reach the rows of adapter 1 alone; a NaN in a row of
    x reaches that row alone."""
    x, w, a, b, _, scales = draw(M, 64, 128, 3, 16, torch.bfloat16, 11)
    a[1, 0, 0], b[1, :, 1], b[1, 3, 2] = math.inf, math.nan, -math.inf
    rows = torch.tensor([i % 4 - 1 for i in range(M)], dtype=torch.int32, device=DEV)
    out = tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales)
    good = (rows != 1).cpu()
    assert torch.isnan(out[~good.to(DEV)]).all()
    check(out[good], x[good], w, a, b, rows[good], scales)
    if M > 4:
        x[5] = math.nan  # (row 5 has adapter 0)
        out2 = tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales)
        keep = good.clone()
        keep[5] = False
        assert torch.isnan(out2[5]).all() and torch.equal(out2[keep], out[keep])


@pytest.mark.parametrize("M", [7, 70])
def test_no_adapters(M):
    """Numbers outside 0 .. L-1, L = 0 and R = 0 all give the projection; K = 0 zeros."""
    x, w, a, b, _, _ = draw(M, 40, 64, 2, 8, torch.float16, 12)
    none = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    far = torch.tensor([2**31 - 1, -2**31, 2, -1, 5, 1000, -7] * M, dtype=torch.int32, device=DEV)[:M]
    p = tcm.lora_gemm_tn(x, w, a, b, none)
    check(p, x, w, a, b, none)
    assert torch.equal(tcm.lora_gemm_tn(x, w, a, b, far), p)
    assert torch.equal(tcm.lora_gemm_tn(x, w, a[:0], b[:0], none), p)
    assert torch.equal(tcm.lora_gemm_tn(x, w, a[:, :0].contiguous(), b[:, :, :0].contiguous(), none), p)
    zero = torch.zeros((M,), dtype=torch.int32, device=DEV)
    e = lambda t: t[..., :0].contiguous()  # noqa: E731
    out = torch.full((M, 40), math.nan, dtype=torch.float16, device=DEV)
    assert (tcm.lora_gemm_tn(e(x), e(w), e(a), b, zero, out=out) == 0).all()
    assert tcm.lora_gemm_tn(x[:0], w, a, b, none[:0]).shape == (0, 40)


def test_same_bits_again_and_from_a_dirty_workspace():
    for M in (1, 48, 130):
        x, w, a, b, rows, scales = draw(M, 96, 2048, 5, 16, torch.bfloat16, 13)
        ws = torch.full((tcm.lora_workspace(M, 2048, 16),), 255, dtype=torch.uint8, device=DEV)  # NaN
        one = tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales, workspace=ws)
        ws.fill_(127)
        assert torch.equal(one, tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales, workspace=ws))
        assert torch.equal(one, tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales))
        with pytest.raises(tcm.TcmError):
            tcm.lora_gemm_tn(x, w, a, b, rows, workspace=ws[: ws.numel() - 16])


def test_row_order_does_not_matter():
    """Each row's result is that of the row alone, to the bits within one size class."""
    x, w, a, b, rows, scales = draw(48, 64, 512, 5, 16, torch.bfloat16, 14)
    perm = torch.randperm(48, generator=torch.Generator().manual_seed(1)).to(DEV)
    out = tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales)
    got = tcm.lora_gemm_tn(x[perm], w, a, b, rows[perm].contiguous(), scales=scales)
    ref, s = ol.lora(f64(x), f64(w), f64(a), f64(b), rows.tolist(), f64(scales))
    tol = 2 * s * (600 * 2.0 ** -24 + 2.0 ** -16) + 2.02 * ol.half_ulp(ref, "bf16")
    assert (np.abs(f64(got) - f64(out[perm])) <= tol[perm.cpu().numpy()]).all()
