"""Heads whose mean of squares lies below fp32's normal numbers (2^-126): norm, rotation and gradients against the
float64 oracle.

The heads hold whole multiples of 2^-66 up to 4 and D is a power of two, so squares, sum and mean are exact in fp32
and what is left are the roundings counted in test_gpu_rope.py.
"""
import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol
from test_gpu_rope import DEV, NAMES, REL, close, f64, freqs, gen, normal, tolerance

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def small(shape, g):
    x = torch.randint(-4, 5, shape, generator=g).double()
    x[..., 0] = 1
    return (x * 2.0 ** -66).to(BF).to(DEV)


@pytest.mark.parametrize("D", [16, 64, 128, 256])
def test_forward(D):
    g = gen(D)
    T, Hq, Hk = 5, 3, 2
    q, k = small((T, Hq, D), g), small((T, Hk, D), g)
    w = normal((D,), g, torch.float32, 0.2, 1.0)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32).to(DEV)
    f = freqs(D)
    outs = tcm.qk_norm_rope(q, k, pos, f, wq=w, wk=w, eps=0.0)
    for x, out in zip((q, k), outs):
        ref = ol.norm_rope(f64(x), pos.tolist(), f64(f), f64(w), 0.0)
        close(out, ref, tolerance(ref, f64(x), f64(f), "half", 1.0, f64(w), True, 0.0), NAMES[BF])


@pytest.mark.parametrize("D", [64, 256])
def test_backward(D):
    g = gen(D + 1)
    T, Hq, Hk = 5, 3, 2
    q, k = small((T, Hq, D), g), small((T, Hk, D), g)
    gq, gk = normal((T, Hq, D), g, BF), normal((T, Hk, D), g, BF)
    w = normal((D,), g, torch.float32, 0.2, 1.0)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32).to(DEV)
    f = freqs(D)
    dq, dk, dwq, dwk = tcm.qk_norm_rope_bwd(gq, gk, q, k, pos, f, wq=w, wk=w, eps=0.0)
    for x, dy, dx, dw in ((q, gq, dq, dwq), (k, gk, dk, dwk)):
        ref, refw, s, sw = ol.norm_rope_bwd(f64(dy), f64(x), pos.tolist(), f64(f), f64(w), 0.0)
        close(dx, ref, REL * s, NAMES[BF])
        assert (np.abs(f64(dw) - refw) <= (REL + 500 * 2.0 ** -24) * sw).all()
