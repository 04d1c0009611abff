"""paged_attention loses nothing but its one rounding to fp32's errors: the tolerance leaves no room
for probabilities of 8 or 11 bits.

A score is an fp32 sum of D products, off by at most (2 D + 8) 2^-24 of the largest sum of
magnitudes of its row, and so is the exponent of its probability, whose exponential adds 2^-20; a
probability enters its product as two values of the type, off by at most 2^-16 (bf16) or 2^-21
(fp16) of itself, half of which is asked of a sum of them, and by 2^-40 of the row's largest
(fp16's smallest number, times 2^-15); its sums are fp32, over at most a tile's 32 keys of a chunk's turns and the
joins; then the output is rounded once.
"""
import math

import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol

DEV = "cuda"
NAMES = {torch.bfloat16: "bf16", torch.float16: "f16"}
STEP = {torch.bfloat16: 2.0 ** -17, torch.float16: 2.0 ** -22}


def f64(t):
    return t.double().cpu().numpy()


def close(out, lse, ref, rlse, mag, top, dtype, D, n, vmax):
    """Raises unless out (and lse) are ref (rlse) but for the errors above; float64 arrays, dtype
    of the output."""
    ds = (2 * D + 8) * 2.0 ** -24 * top + 2.0 ** -20
    rel = STEP[dtype] + 2 * ds[..., None] + (min(n, 1024) // 32 + 300) * 2.0 ** -24
    tol = rel * (mag + np.abs(ref)) + 1.001 * ol.half_ulp(ref, NAMES[dtype])
    if dtype is torch.float16:
        tol = tol + n * 2.0 ** -40 * vmax
    err = np.abs(out - ref)
    assert (err <= tol).all(), f"worst {np.nanmax(err / tol)} at {np.argwhere(~(err <= tol))[:4]}"
    if lse is not None:
        empty = np.isneginf(rlse)
        assert (np.isneginf(lse) == empty).all()
        assert (np.abs(lse[~empty] - rlse[~empty]) <= (ds + 1e-5)[~empty]).all()


def check(q, kc, vc, table, lengths, out, lse, scale, ks=1.0, vs=1.0):
    k, v = f64(kc.float()) * ks, f64(vc.float()) * vs
    ref, rlse, mag, top = ol.paged_attention(f64(q), k, v, table.cpu().numpy(), lengths.tolist(), kc.shape[1], scale)
    close(f64(out), None if lse is None else f64(lse), ref, rlse, mag, top, q.dtype, q.shape[-1],
          int(max(lengths.tolist())), np.abs(v).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 2, 64), (32, 8, 128), (20, 1, 96), (4, 2, 256), (3, 3, 144), (6, 2, 32)])
def test_one_rounding(Hq, Hk, D, page, kind, dt):
    from test_gpu_paged_attention import make

    q, kc, vc, table, n = make(6, Hq, Hk, D, [1, 8, 40, 300, 2, 5000], page, dt, kind, Hq + D)
    # scores of about 1, so that their own errors leave the rest to be seen
    scale = 0.125 * D ** -0.5 / (16 if kind == "e4m3" else 1)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float32, device=DEV)
    kw = dict(k_scale=0.5, v_scale=0.25) if kind == "e4m3" else {}
    out = tcm.paged_attention(q, kc, vc, table, n, scale=scale, lse=lse, **kw)
    check(q, kc, vc, table, n, out, lse, scale, kw.get("k_scale", 1.0), kw.get("v_scale", 1.0))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("n", [1, 40, 3000])
def test_infinite_values(n, page, dt):
    """An attended infinity is the result's (of both signs: NaN); NaN is too; the other elements and the
    other sequence are as they were."""
    from test_gpu_paged_attention import make

    D = 64
    case = q, kc, vc, table, lengths = make(2, 4, 2, D, [n, n], page, dt, seed=n)
    want = tcm.paged_attention(*case)
    spoilt = vc.clone()
    at = lambda j: (int(table[0, j // page]), j % page, 0)  # noqa: E731
    first, last = at(n // 2), at(n - 1)
    spoilt[first][3], spoilt[last][20] = math.inf, -math.inf
    spoilt[first][33], spoilt[first][50], spoilt[last][50] = math.nan, math.inf, -math.inf
    out = tcm.paged_attention(q, kc, spoilt, table, lengths)
    assert torch.isposinf(out[0, :2, 3]).all() and torch.isneginf(out[0, :2, 20]).all()
    assert torch.isnan(out[0, :2, 33]).all()
    assert (torch.isneginf(out[0, :2, 50]) if first == last else torch.isnan(out[0, :2, 50])).all()
    rest = [d for d in range(D) if d not in (3, 20, 33, 50)]
    step = 2.0 ** (-8 if dt is torch.bfloat16 else -11)  # (room for a form that rounds probabilities once)
    size = want.float().abs().max()
    assert ((out[0, :2, rest].float() - want[0, :2, rest].float()).abs() <= 2 * step * size).all()
    assert torch.equal(out[0, 2:], want[0, 2:]) and torch.equal(out[1], want[1])
