"""The operators of a step that drafts from their definitions, in numpy float64 (whole numbers:
plain Python) on the CPU.  Shares nothing with the GPU path; next to each result stands what
its rounding errors scale with.
"""
from __future__ import annotations

import numpy as np


def add_rms_norm(x, r=None, w=None, eps=1e-6):
    """(y, s): s = x + r, y = w s / sqrt(mean(s^2) + eps)"""
    s = x if r is None else x + r
    y = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return (y if w is None else y * w), s


def add_rms_norm_bwd(dy, s, w=None, ds=None, eps=1e-6):
    """(dx, dw, scale of dx's errors, scale of dw's)"""
    f = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    h = s * f
    g = dy if w is None else dy * w
    dx = f * (g - h * (g * h).mean(-1, keepdims=True))
    mag = f * (np.abs(g) + np.abs(h) * np.abs(g * h).mean(-1, keepdims=True))
    if ds is not None:
        dx, mag = dx + ds, mag + np.abs(ds)
    return dx, (dy * h).sum(0), mag, np.abs(dy * h).sum(0)


def mx_exponents(y):
    """The smallest e >= -127 with |element| <= 448 * 2^e for the finite ones of each 32 of y (T, D):
    (T, D / 32)"""
    top = np.abs(np.where(np.isfinite(y), y, 0.0)).reshape(y.shape[0], -1, 32).max(-1)
    m, e = np.frexp(top)  # 448 = 0.875 * 2^9
    return np.where(top == 0, -127, np.maximum(e - 9 + (m > 0.875), -127))


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def nibbles(w):
    """The 4-bit elements of (N, K / 2) bytes: (N, K)"""
    return np.stack([w & 15, w >> 4], -1).reshape(w.shape[0], -1)


def gemm_w4(x, w, scales, zeros=None, elem="u4"):
    """(out, s): x W^T and the sums that its errors scale with; scales as stored (E8M0 bytes for "e2m1")"""
    q = nibbles(w)
    group = q.shape[1] // max(scales.shape[1], 1) if q.shape[1] else 1
    if elem == "e2m1":
        f = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
        v = E2M1[q] * np.repeat(f, group, 1)
        return x @ v.T, np.abs(x) @ np.abs(v).T
    f = np.repeat(scales.astype(np.float64), group, 1)
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, 1)
    return x @ ((q - z) * f).T, np.abs(x) @ ((q + z) * np.abs(f)).T


def sees(i, j, context, bits, window, tokens):
    """Does token i of a sequence's `tokens` see key j?  bits: its row as a Python int, None in a chain."""
    if bits is None:
        return j <= context + i and not (window and j <= context + i - window)
    if j >= context:
        return bits >> (j - context) & 1 == 1
    depth = bin(bits & ((1 << tokens) - 1)).count("1")
    return not (window and j <= context + depth - 1 - window)


def tree_attention(q, k, v, table, lengths, starts, page_size, scale, tree=None, window=0, max_nodes=None):
    """{row: (out (Hq, D), lse (Hq,), sum_j p_j |v_j|, largest scale sum_d |q_d k_d|)} for the rows of q
    (T, Hq, D) that are computed; tree: a Python int a row."""
    T, Hq, D = q.shape
    pages = k.shape[0]
    G = Hq // k.shape[2]
    done = {}
    for b in range(len(lengths)):
        m = int(starts[b + 1]) - int(starts[b])
        n = min(max(int(lengths[b]), 0), table.shape[1] * page_size)
        context = max(0, n - m)
        for i in range(m if max_nodes is None else min(m, max_nodes)):
            t = int(starts[b]) + i
            if t >= T:
                break
            keys = [j for j in range(n) if 0 <= table[b, j // page_size] < pages and
                    sees(i, j, context, None if tree is None else tree[t], window, m)]
            out, mag = np.zeros((Hq, D)), np.zeros((Hq, D))
            lse, top = np.full(Hq, -np.inf), np.zeros(Hq)
            if keys:
                pg = np.array([table[b, j // page_size] for j in keys])
                at = np.array([j % page_size for j in keys])
                for h in range(Hq):
                    kk, vv = k[pg, at, h // G], v[pg, at, h // G]
                    s = scale * (kk @ q[t, h])
                    e = np.exp(s - s.max())
                    lse[h] = s.max() + np.log(e.sum())
                    e /= e.sum()
                    out[h], mag[h] = e @ vv, e @ np.abs(vv)
                    top[h] = (abs(scale) * (np.abs(kk) @ np.abs(q[t, h]))).max()
            done[t] = out, lse, mag, top
    return done


def cache_plan(lengths, change, table, stack, count, page_size, T, pages):
    """(lengths, table, stack, count, starts, slots, positions, missing) after the change; lists in, lists out"""
    lengths, table, stack = list(lengths), [list(r) for r in table], list(stack)
    count = min(max(count, 0), len(stack))
    room = len(table[0]) * page_size if table else 0
    span = []
    returned = []
    for b, n in enumerate(lengths):
        n = min(max(n, 0), room)
        end = min(max(n + change[b], 0), room)
        span.append((n, end))
        for e in range(-(-end // page_size), -(-n // page_size)):
            if 0 <= table[b][e] < pages:
                returned.append(table[b][e])
            table[b][e] = -1
    for r, page in enumerate(returned):
        at = count + len(returned) - 1 - r
        if at < len(stack):
            stack[at] = page
    top = min(count + len(returned), len(stack))
    taken = 0
    for b, (n, end) in enumerate(span):
        for e in range(-(-n // page_size), -(-end // page_size)):
            at = top - 1 - taken
            table[b][e] = stack[at] if at >= 0 else -1
            taken += 1
    starts, slots, positions = [0], [], []
    for b, (n, end) in enumerate(span):
        for key in range(n, end):
            page = table[b][key // page_size]
            slots.append(page * page_size + key % page_size if 0 <= page < pages else -1)
            positions.append(key)
        starts.append(len(slots))
    pad = max(0, T - len(slots))
    return ([e for _, e in span], table, stack, max(top - taken, 0), starts, (slots + [-1] * pad)[:T],
            (positions + [0] * pad)[:T], max(taken - top, 0))
