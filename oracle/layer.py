"""The layer operators from their definitions, in numpy float64 on the CPU.

Shares nothing with the GPU path: inputs are float64 arrays of the values the stored
elements stand for, loops run over rows, heads and keys, and next to each result
stands what its rounding errors scale with.
"""
from __future__ import annotations

import numpy as np


def half_ulp(x, dtype):
    """Half the spacing of `dtype` ("bf16", "f16", "f32", "e4m3") at |x|: the most a
    rounding to nearest moves a value of its range."""
    bits, low = {"bf16": (8, -126), "f16": (11, -14), "f32": (24, -126), "e4m3": (4, -6)}[dtype]
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** low)))
    return 2.0 ** (np.maximum(e, low) - bits)


def lora(x, w, a, b, rows, scales=None, ranks=None):
    """(out, s): out[i] = x[i] w^T + scales[r] (x[i] a_r^T) b_r^T, r = rows[i] (outside
    0 .. L-1: the first term), and the same sums of magnitudes."""
    L, R = a.shape[:2]
    out = x @ w.T
    s = np.abs(x) @ np.abs(w).T
    for i, r in enumerate(rows):
        if 0 <= r < L:
            n = R if ranks is None else min(max(int(ranks[r]), 0), R)
            f = 1.0 if scales is None else float(scales[r])
            ar, br = a[r, :n], b[r, :, :n]
            out[i] += f * (br @ (ar @ x[i]))
            s[i] += abs(f) * (np.abs(br) @ (np.abs(ar) @ np.abs(x[i])))
    return out, s


def _pairs(rot, layout):
    j = np.arange(rot // 2)
    return (j, j + rot // 2) if layout == "half" else (2 * j, 2 * j + 1)


def rotate(n, positions, inv_freq, layout, factor=1.0, back=False):
    """n (T, H, D) with the pairs of its first 2 len(inv_freq) elements turned by
    positions[t] * inv_freq[j] (back: by the negative) and scaled by factor."""
    y = n.copy()
    lo, hi = _pairs(2 * len(inv_freq), layout)
    for t, p in enumerate(positions):
        # the angle as whole turns and the rest: exact for the sizes used here
        angle = np.remainder(np.longdouble(int(p)) * inv_freq.astype(np.longdouble),
                             2 * np.longdouble("3.14159265358979323846264338327950288"))
        c, s = np.cos(angle).astype(np.float64), np.sin(angle).astype(np.float64)
        s = -s if back else s
        y[t, :, lo] = (factor * (n[t][:, lo] * c - n[t][:, hi] * s)).T
        y[t, :, hi] = (factor * (n[t][:, hi] * c + n[t][:, lo] * s)).T
    return y


def norm_rope(x, positions, inv_freq, w=None, eps=1e-6, layout="half", factor=1.0, norm=True):
    """rotate(x w / sqrt(mean(x^2) + eps))"""
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if w is not None:
            x = x * w
    return rotate(x, positions, inv_freq, layout, factor)


def norm_rope_bwd(dy, x, positions, inv_freq, w=None, eps=1e-6, layout="half", factor=1.0, norm=True):
    """(dx, dw, scale of dx's errors, scale of dw's)"""
    dn = rotate(dy, positions, inv_freq, layout, factor, back=True)
    mag = np.abs(factor) * np.abs(dy).max(-1, keepdims=True) + np.abs(dn)
    if not norm:
        return dn, None, mag, None
    g = dn if w is None else dn * w
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = x * r
    dx = r * (g - h * (g * h).mean(-1, keepdims=True))
    wm = 1.0 if w is None else np.abs(w)
    s = r * (mag * wm + np.abs(h) * (mag * wm * np.abs(h)).mean(-1, keepdims=True))
    return dx, (dn * h).sum((0, 1)), s, (mag * np.abs(h)).sum((0, 1))


def paged_attention(q, k, v, table, lengths, page_size, scale, window=0, pages=None):
    """(out, lse, a, x): attention of q (B, Hq, D) over caches k, v (pages, page_size,
    Hk, D), its log sum of exponentials, sum_j p_j |v_j| (B, Hq, D) and the largest
    scale sum_d |q_d k_d| of a row (B, Hq)."""
    B, Hq, D = q.shape
    pages = k.shape[0] if pages is None else pages
    G = Hq // k.shape[2]
    out = np.zeros((B, Hq, D))
    mag = np.zeros((B, Hq, D))
    lse = np.full((B, Hq), -np.inf)
    top = np.zeros((B, Hq))
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * page_size)
        keys = [j for j in range(max(0, n - window) if window else 0, n)
                if 0 <= table[b, j // page_size] < pages]
        if not keys:
            continue
        pg = np.array([table[b, j // page_size] for j in keys])
        at = np.array([j % page_size for j in keys])
        for h in range(Hq):
            kk, vv = k[pg, at, h // G], v[pg, at, h // G]
            s = scale * (kk @ q[b, h])
            m = s.max()
            p = np.exp(s - m)
            lse[b, h] = m + np.log(p.sum())
            p /= p.sum()
            out[b, h] = p @ vv
            mag[b, h] = p @ np.abs(vv)
            top[b, h] = (abs(scale) * (np.abs(kk) @ np.abs(q[b, h]))).max()
    return out, lse, mag, top
