"""paged_tree_attention where a row's largest score is above others by more than fp32 holds of a probability: what is
finite vanishes, however large, and an infinite value is one or NaN in its own element alone, wherever tiles, waves and
parts join.

One key has a score of its own and the others 0.  With 400 (577 in base 2) every other probability is 0 in any precision
here, and the exact result is that key's value; with 14 (20 in base 2) all count.
"""
import math

import pytest
import torch

import tensor_core_matrix_amd as tcm
from test_gpu_tree_attention import BF, DEV, HF

pytestmark = pytest.mark.gpu


def call(n, m, far, values, dt, G=1, D=64, page=16, score=400):
    """m tokens in a row on n keys of a sequence, whose key `far` has this score and the others 0; values: {(key,
    element): value}, 1 elsewhere at key `far`, 0.5 at the others."""
    pages = -(-n // page)
    k = torch.zeros((pages, page, 1, D), dtype=dt, device=DEV)
    v = torch.full_like(k, 0.5)
    k[far // page, far % page, 0, 0] = score / 8
    v[far // page, far % page, 0] = 1.0
    for (key, d), x in values.items():
        v[key // page, key % page, 0, d] = x
    q = torch.zeros((m, G, D), dtype=dt, device=DEV)
    q[:, :, 0] = 8.0
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    lse = torch.empty((m, G), dtype=torch.float32, device=DEV)
    out = tcm.paged_tree_attention(q, k, v, i32(*range(pages)).view(1, -1), i32(n), i32(0, m), m, scale=1.0, lse=lse)
    assert score < 400 or ((lse - 400).abs() < 1e-3).all()  # (an fp32 of 577 in base 2 is off by 3e-5)
    return out


# (n, m, G): few rows, whose waves take tiles in turn; more; 128 rows; one stretch or many
SHAPES = [(100, 2, 1), (300, 2, 1), (300, 20, 1), (300, 20, 4), (700, 33, 4), (6000, 2, 1), (6000, 20, 1), (6000, 20, 4)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,m,G", SHAPES)
def test_finite_values_vanish(n, m, G, D):
    """bf16 values up to the type's largest, before and behind the key that counts (one an element: two of them pass
    what an fp32 sum holds)."""
    big = torch.finfo(BF).max
    for far in (n // 2, n - m, 40):
        values = {(key, d): x for key, d, x in ((0, 3, big), (7, 5, -big), (33, 6, big), (39, 7, 2.0 ** 100), (n // 3, 8, big))
                  if key != far}
        assert (call(n, m, far, values, BF, G, D) == 1).all(), far


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("n,m,G", SHAPES)
def test_infinite_values(n, m, G, D, dt):
    """At the first key, and the largest score in a later tile: infinite while the probability is a number (2^-20 here),
    and not finite when it is none."""
    for far in {max(70, n // 2), n - m}:
        odd = {(0, 3): math.inf, (0, 9): -math.inf, (0, 17): math.nan}
        rest = [d for d in range(D) if d not in (3, 9, 17)]
        out, clean = call(n, m, far, odd, dt, G, D, score=14), call(n, m, far, {}, dt, G, D, score=14)
        assert (out[..., 3] == math.inf).all() and (out[..., 9] == -math.inf).all(), far
        assert torch.isnan(out[..., 17]).all() and torch.equal(out[..., rest], clean[..., rest])
        out = call(n, m, far, odd, dt, G, D)
        assert not torch.isfinite(out[..., [3, 9, 17]]).any() and (out[..., rest] == 1).all(), far
