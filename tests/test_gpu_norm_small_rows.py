"""Rows whose mean of squares lies below fp32's normal numbers (2^-126): the norm, its MXFP8 form and its
gradients against the float64 oracle.

The rows hold whole multiples of 2^-66 up to 4 and D is a power of two, so the squares (multiples of 2^-132), their sum
and the mean (a multiple of 2^-147) are exact in fp32 and what is left are the roundings counted in test_gpu_norm.py.
"""
import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import step as os_
from test_gpu_norm import BF, DEV, F32, R, check_mx, f64, rand, weight, within

pytestmark = pytest.mark.gpu


def small(T, D, seed, step=2.0 ** -66):
    """Multiples of `step` from -4 to 4, the first of each row not zero"""
    x = torch.randint(-4, 5, (T, D), generator=torch.Generator().manual_seed(seed)).double()
    x[:, 0] = 1
    return (x * step).to(BF).to(DEV)


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140])
@pytest.mark.parametrize("step", [2.0 ** -66, 2.0 ** -64, 2.0 ** -60])
@pytest.mark.parametrize("D", [8, 512, 2048, 4096, 8192, 32768])
def test_norm(D, step, eps):
    T = 5
    x = small(T, D, D, step)
    w = weight("f32", D, BF)
    for r in (None, small(T, D, D + 1, step)):
        for odt in (BF, F32):
            y, s = tcm.add_rms_norm(x, w, r, eps=eps, out_dtype=odt)
            ref, total = os_.add_rms_norm(f64(x), None if r is None else f64(r), f64(w), eps)
            within(y, ref, R * np.abs(ref) + 1e-37, odt)
            within(s, total, 2.0 ** -23 * np.abs(total), BF)


def test_a_row_of_zeros_with_the_least_eps():
    x = torch.zeros((3, 512), dtype=BF, device=DEV)
    for eps in (2.0 ** -149, 2.0 ** -140, 2.0 ** -127, 2.0 ** -126):
        assert (tcm.add_rms_norm(x, eps=eps)[0] == 0).all(), eps
        dx, dw = tcm.add_rms_norm_bwd(torch.zeros_like(x), x, weight("f32", 512, BF), eps=eps)
        assert (dx == 0).all() and (dw == 0).all(), eps


@pytest.mark.parametrize("D", [512, 4096])
def test_mx(D):
    x = small(4, D, 7)
    q, e, s = tcm.add_rms_norm_mx_fp8(x, eps=2.0 ** -149)
    # (2^-149 is 2^-15 of the mean or less, and the sum is exact: multiples of 2^-149)
    ref, _ = os_.add_rms_norm(f64(x), eps=2.0 ** -149)
    f = np.repeat(2.0 ** (e.cpu().numpy().astype(int) - 127.0), 32, 1)
    v = f64(q.float()) * f
    assert np.isfinite(v).all() and (np.abs(v - ref) <= 2.0 ** -4 * np.abs(ref) + 2.0 ** -9 * f).all()
    check_mx(x * 2.0 ** 60, None, None, *tcm.add_rms_norm_mx_fp8(x * 2.0 ** 60))


@pytest.mark.parametrize("D", [512, 2048, 8192, 32768])
def test_gradients(D):
    T = 6
    s, dy, w = small(T, D, D), rand((T, D), 2, BF), weight("f32", D, BF)
    dx, dw = tcm.add_rms_norm_bwd(dy, s, w, eps=0.0)
    rx, rw, mx, mw = os_.add_rms_norm_bwd(f64(dy), f64(s), f64(w), eps=0.0)
    within(dx, rx, 2 * R * mx, BF)
    assert (np.abs(f64(dw) - rw) <= (48 + 64) * 2.0 ** -24 * mw + 1e-30).all()
