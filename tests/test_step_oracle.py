"""The float64 definitions that the GPU tests of a drafting step compare with, against independent
statements of the same: differences, dense torch forms, an undone plan (CPU)."""
import math
import random

import numpy as np
import pytest
import torch

from oracle import layer as ol
from oracle import step as os_


@pytest.mark.parametrize("weighted", [False, True])
def test_norm_gradients_against_differences(weighted):
    g = np.random.default_rng(1)
    s, dy, ds = g.normal(size=(3, 5, 16))
    w = 1 + 0.3 * g.normal(size=16) if weighted else None
    dx, dw, _, _ = os_.add_rms_norm_bwd(dy, s, w, ds, eps=1e-3)
    loss = lambda s_, w_: (os_.add_rms_norm(s_, None, w_, 1e-3)[0] * dy).sum() + (s_ * ds).sum()  # noqa: E731
    step = 1e-5
    for t, d in ((3, 7), (0, 0), (4, 15)):
        p, m = s.copy(), s.copy()
        p[t, d] += step
        m[t, d] -= step
        assert abs((loss(p, w) - loss(m, w)) / (2 * step) - dx[t, d]) < 1e-7
    if weighted:
        for d in (0, 9):
            p, m = w.copy(), w.copy()
            p[d] += step
            m[d] -= step
            assert abs((loss(s, p) - loss(s, m)) / (2 * step) - dw[d]) < 1e-7


def test_norm_against_torch():
    g = torch.Generator().manual_seed(2)
    x, r = torch.randn((2, 7, 24), generator=g, dtype=torch.float64)
    w = torch.randn(24, generator=g, dtype=torch.float64)
    y, s = os_.add_rms_norm(x.numpy(), r.numpy(), w.numpy(), 1e-5)
    ref = torch.nn.functional.rms_norm(x + r, (24,), w, 1e-5)
    assert np.abs(y - ref.numpy()).max() < 1e-13 and (s == (x + r).numpy()).all()


def test_mx_exponents():
    y = np.zeros((1, 32 * 6))
    y[0, 0], y[0, 32], y[0, 64], y[0, 96], y[0, 128] = 448, 448.0001, -1, np.inf, 2.0 ** -140
    y[0, 97] = 3.5
    # 1 <= 448 * 2^-8 = 1.75 and more than 0.875; 3.5 = 448 * 2^-7
    assert os_.mx_exponents(y).tolist() == [[0, 1, -8, -7, -127, -127]]


def test_w4_values():
    w = np.array([[0x10, 0xF8] + [0] * 14], dtype=np.uint8)
    x = np.eye(32)[:4]
    out, _ = os_.gemm_w4(x, w, np.array([[2.0]]), np.array([[3]]))
    assert out[:, 0].tolist() == [2 * (q - 3) for q in (0, 1, 8, 15)]
    out, _ = os_.gemm_w4(x, w, np.array([[126]], dtype=np.uint8), elem="e2m1")
    assert out[:, 0].tolist() == [0, 0.25, 0, -3]


@pytest.mark.parametrize("window", [0, 1, 4, 9])
def test_a_chain_is_one_token_at_a_time(window):
    """Token i of a chain is one new token of a sequence that ends with it; so is a path of a tree."""
    g = np.random.default_rng(3)
    Hq, Hk, D, page, n, m = 4, 2, 8, 4, 14, 5
    k, v = g.normal(size=(2, 6, page, Hk, D))
    table = np.array([[3, 0, 5, 1]])
    q = g.normal(size=(m, Hq, D))
    got = os_.tree_attention(q, k, v, table, [n], [0, m], page, 0.4, None, window)
    path = os_.tree_attention(q, k, v, table, [n], [0, m], page, 0.4, [(2 << i) - 1 for i in range(m)], 0)
    for i in range(m):
        out, lse, _, _ = ol.paged_attention(q[i:i + 1], k, v, table, [n - m + 1 + i], page, 0.4, window)
        assert np.abs(got[i][0] - out[0]).max() < 1e-14 and np.abs(got[i][1] - lse[0]).max() < 1e-14
        if not window:
            assert np.abs(path[i][0] - out[0]).max() < 1e-14


def test_a_tree_against_a_dense_mask():
    g = torch.Generator().manual_seed(4)
    n, m, D = 12, 4, 8
    k, v = torch.randn((2, 3, 4, 1, D), generator=g, dtype=torch.float64)
    q = torch.randn((m, 1, D), generator=g, dtype=torch.float64)
    bits = [0b0001, 0b0011, 0b0101, 0b1101]
    for window in (0, 3):
        mask = torch.zeros((m, n), dtype=torch.bool)
        for i in range(m):
            depth = bin(bits[i]).count("1")  # the token is at place 8 + depth - 1
            for j in range(n):
                mask[i, j] = bool(bits[i] >> (j - 8) & 1) if j >= 8 else not window or 8 + depth - 1 - j < window
        ref = torch.nn.functional.scaled_dot_product_attention(
            q[:, 0], k[[2, 0, 1]].reshape(12, D), v[[2, 0, 1]].reshape(12, D), mask)
        got = os_.tree_attention(q.numpy(), k.numpy(), v.numpy(), np.array([[2, 0, 1]]), [n], [0, m], 4,
                                 1 / math.sqrt(D), bits, window)
        assert np.abs(np.stack([got[i][0][0] for i in range(m)]) - ref.numpy()).max() < 1e-12


@pytest.mark.parametrize("seed", range(20))
def test_a_plan_undone(seed):
    r = random.Random(seed)
    page, per, B = r.choice([1, 3, 16]), 8, r.randrange(1, 9)
    lengths = [r.randrange(0, per * page // 2 + 1) for _ in range(B)]
    order = r.sample(range(B * per), B * per)
    table = [[order.pop() if e * page < n else -1 for e in range(per)] for n in lengths]
    stack, count = order + [-1] * (B * per - len(order)), len(order)
    change = [r.randrange(-n, per * page - n + 1) for n in lengths]
    a = os_.cache_plan(lengths, change, table, stack, count, page, 10000, B * per)
    held = [p for row in a[1] for p in row if p >= 0] + a[2][:a[3]]
    assert sorted(held) == list(range(B * per)) and a[7] == 0
    used = [s for s in a[5] if s >= 0]
    assert len(set(used)) == len(used) == sum(max(0, c) for c in change) == a[4][-1]
    b = os_.cache_plan(a[0], [-c for c in change], a[1], a[2], a[3], page, 0, B * per)
    assert b[0] == lengths and b[1] == table and b[2][:count] == stack[:count] and b[3] == count
