"""qk_norm_rope, qk_norm_rope_cache and qk_norm_rope_bwd on the GPU against the float64
oracle.

Tolerance: everything is computed in fp32 from exact inputs.  The norm's factor is off
by at most (D / 2 + 4) 2^-24 of itself, the cosine and sine by 4e-7 (an angle rounded once
to fp32 after its reduction in 64 bits), each product and sum by 2^-24: 3e-5 of the
magnitudes involved covers D = 256.  The result is rounded once (half an ulp).
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
REL = 3e-5


def f64(t):
    return t.double().cpu().numpy()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(shape, g, dt, sigma=1.0, mean=0.0):
    return (mean + sigma * torch.randn(shape, generator=g)).to(dt).to(DEV)


def freqs(rot):
    return tcm.rope_frequencies(rot, device=DEV)[0]


def tolerance(ref, x, inv_freq, layout, factor, w=None, norm=True, eps=1e-6):
    """REL of the magnitudes a rotated pair is made of."""
    n = ol.norm_rope(x, [0] * x.shape[0], inv_freq, w, eps, layout, 1.0, norm)
    m = np.abs(n)
    lo, hi = ol._pairs(2 * len(inv_freq), layout)
    both = m[..., lo] + m[..., hi]
    m[..., lo] = m[..., hi] = abs(factor) * both
    return REL * m


def close(out, ref, tol, dtype):
    err = np.abs(f64(out) - ref)
    t = tol + 1.01 * ol.half_ulp(np.abs(ref) + tol, dtype)
    assert (err <= t).all(), f"worst {np.nanmax(err / t)} at {np.argwhere(~(err <= t))[:4]}"


SHAPES = [  # T, Hq, Hk, D, rot
    (1, 1, 1, 8, 8), (1, 32, 8, 128, 128), (3, 5, 2, 64, 64), (2, 4, 4, 64, 32), (7, 3, 1, 80, 80),
    (5, 8, 2, 80, 20), (4, 6, 3, 96, 24), (2, 2, 1, 256, 256), (9, 7, 7, 136, 64), (3, 2, 2, 248, 2),
    (6, 4, 1, 128, 0), (300, 2, 1, 64, 16), (1500, 12, 4, 32, 32), (2, 100, 3, 128, 64),
]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dt, layout):
    T, Hq, Hk, D, rot = shape
    g = gen(sum(shape))
    qkv = normal((T, (Hq + Hk) * D), g, dt, 2.0)
    q, k = qkv.view(T, Hq + Hk, D).split([Hq, Hk], 1)  # views of a fused projection
    wq, wk = normal((D,), g, dt, 0.2, 1.0), normal((D,), g, dt, 0.2, 1.0)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32).to(DEV)
    pos[0] = 2**31 - 1
    f = freqs(rot) if rot else None
    ff = f64(f) if rot else np.zeros(0)
    for norm, factor in ((True, 1.0), (False, 1.25)):
        w = dict(wq=wq, wk=wk) if norm else {}
        qo, ko = tcm.qk_norm_rope(q, k, pos, f, **w, eps=1e-5, layout=layout, factor=factor, norm=norm)
        for x, o, wt in ((q, qo, wq), (k, ko, wk)):
            wt = f64(wt) if norm else None
            ref = ol.norm_rope(f64(x), pos.tolist(), ff, wt, 1e-5, layout, factor, norm)
            close(o, ref, tolerance(ref, f64(x), ff, layout, factor, wt, norm, 1e-5), NAMES[dt])


def test_weights_of_32_bits_none_and_one():
    g = gen(5)
    q, k = normal((6, 4, 64), g, torch.bfloat16), normal((6, 2, 64), g, torch.bfloat16)
    pos, f = torch.arange(6, dtype=torch.int32, device=DEV), freqs(64)
    w = normal((64,), g, torch.float32, 0.3, 1.0)
    for wq, wk in ((w, None), (None, w), (None, None)):
        qo, ko = tcm.qk_norm_rope(q, k, pos, f, wq, wk)
        for x, o, wt in ((q, qo, wq), (k, ko, wk)):
            wt = None if wt is None else f64(wt)
            ref = ol.norm_rope(f64(x), pos.tolist(), f64(f), wt)
            close(o, ref, tolerance(ref, f64(x), f64(f), "half", 1.0, wt), "bf16")


def test_in_place_and_strided_outputs():
    g = gen(6)
    T, Hq, Hk, D = 37, 6, 2, 128
    qkv = normal((T, Hq + 2 * Hk, D), g, torch.bfloat16)
    pos, f = torch.arange(T, dtype=torch.int32, device=DEV), freqs(D)
    q, k, v = qkv.split([Hq, Hk, Hk], 1)
    qo, ko = tcm.qk_norm_rope(q, k, pos, f)
    heads_first = torch.empty((Hq, T, D), dtype=torch.bfloat16, device=DEV)
    tcm.qk_norm_rope(q, k, pos, f, q_out=heads_first.transpose(0, 1))
    assert torch.equal(heads_first.transpose(0, 1), qo)
    keep = v.clone()
    tcm.qk_norm_rope(q, k, pos, f, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, keep)


def test_rows_of_zeros_infinities_and_nan():
    """A zero head stays zero; what is not finite stays within its head."""
    g = gen(7)
    q, k = normal((4, 3, 64), g, torch.float16), normal((4, 1, 64), g, torch.float16)
    pos, f = torch.arange(4, dtype=torch.int32, device=DEV), freqs(64)
    want, _ = tcm.qk_norm_rope(q, k, pos, f)
    q2 = q.clone()
    q2[0, 0], q2[1, 1, 3], q2[2, 2, 5] = 0.0, math.nan, math.inf
    got, _ = tcm.qk_norm_rope(q2, k, pos, f)
    assert (got[0, 0] == 0).all() and torch.isnan(got[1, 1]).all() and torch.isnan(got[2, 2]).any()
    for t, h in ((0, 0), (1, 1), (2, 2)):
        got[t, h] = want[t, h]
    assert torch.equal(got, want)


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,page", [(1, 4, 1, 64, 64, 16), (13, 8, 2, 128, 128, 1), (70, 3, 3, 80, 20, 5),
                                               (600, 2, 1, 96, 48, 64), (33, 0, 2, 64, 64, 16)])
def test_into_cache(T, Hq, Hk, D, rot, page, kind, heads_first):
    g = gen(T + D)
    dt = torch.bfloat16
    qkv = normal((T, Hq + 2 * Hk, D), g, dt, 3.0)
    q, k, v = qkv.split([Hq, Hk, Hk], 1)
    pages = -(-T // page) + 2
    shape = (pages, Hk, page, D) if heads_first else (pages, page, Hk, D)
    fill = 0x55
    caches = []
    for _ in range(2):
        c = torch.full((math.prod(shape) * (1 if kind == "e4m3" else 2),), fill, dtype=torch.uint8, device=DEV)
        c = c.view(torch.float8_e4m3fn if kind == "e4m3" else dt).view(shape)
        caches.append(c.transpose(1, 2) if heads_first else c)
    kc, vc = caches
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    slots[T // 2] = -1
    if T > 10:
        slots[3], slots[7] = pages * page, 2**31 - 1
    sl = slots.tolist()
    slots = slots.to(DEV)
    pos = torch.randint(0, 5000, (T,), generator=g).to(torch.int32).to(DEV)
    wq, wk, f = normal((D,), g, dt, 0.1, 1.0), normal((D,), g, dt, 0.1, 1.0), freqs(rot)
    ks, vs = (0.03, 0.0125) if kind == "e4m3" else (1.0, 1.0)
    qo = tcm.qk_norm_rope_cache(q, k, v, pos, f, kc, vc, slots, wq, wk, k_scale=ks, v_scale=vs)
    if Hq:
        ref = ol.norm_rope(f64(q), pos.tolist(), f64(f), f64(wq))
        close(qo, ref, tolerance(ref, f64(q), f64(f), "half", 1.0, f64(wq)), "bf16")
    kr = ol.norm_rope(f64(k), pos.tolist(), f64(f), f64(wk))
    kt = tolerance(kr, f64(k), f64(f), "half", 1.0, f64(wk))
    used = np.zeros((pages * page,), bool)
    for t, s in enumerate(sl):
        if not 0 <= s < pages * page:
            continue
        used[s] = True
        for c, ref, tol, scale in ((kc, kr[t], kt[t], ks), (vc, f64(v)[t], 0 * kt[t], vs)):
            got = c[s // page, s % page]
            if kind == "e4m3":
                scale = float(np.float32(scale))
                want = np.clip(ref / scale, -448, 448)
                close(got.to(torch.float32), want, tol / scale + 1e-6 * np.abs(want), "e4m3")
            else:
                close(got, ref, tol, "bf16")
    for c in (kc, vc):  # slots that no token named are as they were
        raw = c.contiguous().view(torch.uint8).view(pages * page, -1).cpu().numpy()
        assert (raw[~used] == fill).all()


def test_e4m3_saturates_keeps_nan_and_rounds_to_even():
    """Every bf16 value of a sweep of the range, ties among them, as torch rounds it."""
    x = torch.arange(-2**15, 2**15, 8, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[: x.numel() // 64 * 64].view(-1, 1, 64).to(DEV)
    T = x.shape[0]
    kc = torch.zeros((T, 1, 1, 64), dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    tcm.qk_norm_rope_cache(x, x, x, None, None, kc, vc, slots, norm=False)
    want = x.float().clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    for c in (kc, vc):
        got = c.view(torch.float8_e4m3fn).view(-1).float()
        assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(want.view(-1).float(), nan=1e9))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dt, layout):
    T, Hq, Hk, D, rot = shape
    g = gen(sum(shape) + 1)
    qkv = normal((T, (Hq + Hk) * D), g, dt, 2.0)
    q, k = qkv.view(T, Hq + Hk, D).split([Hq, Hk], 1)
    gq, gk = normal((T, Hq, D), g, dt), normal((T, Hk, D), g, dt)
    wq, wk = normal((D,), g, dt, 0.2, 1.0), normal((D,), g, dt, 0.2, 1.0)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32).to(DEV)
    f = freqs(rot) if rot else None
    ff = f64(f) if rot else np.zeros(0)
    for norm, factor in ((True, 0.8), (False, 1.0)):
        w = dict(wq=wq, wk=wk) if norm else {}
        dq, dk, dwq, dwk = tcm.qk_norm_rope_bwd(gq, gk, q, k, pos, f, **w, eps=1e-5, layout=layout, factor=factor,
                                                norm=norm)
        for x, dy, wt, dx, dw in ((q, gq, wq, dq, dwq), (k, gk, wk, dk, dwk)):
            ref, refw, s, sw = ol.norm_rope_bwd(f64(dy), f64(x), pos.tolist(), ff, f64(wt) if norm else None, 1e-5,
                                                layout, factor, norm)
            close(dx, ref, REL * s, NAMES[dt])
            if norm:
                # (a lane's sum of at most T H terms and the tree above it, and what each term is off)
                depth = min(T * x.shape[1], 400) + 100
                assert (np.abs(f64(dw) - refw) <= (REL + depth * 2.0 ** -24) * sw).all()
            else:
                assert dw is None


def test_backward_against_differences_of_the_forward_definition():
    """Along random directions: the gradients' product with a direction is the change of
    the loss <dy, y> that the float64 forward gives.  fp16 gradients are off by half an
    ulp an element; along a random direction their errors are independent: 6 sigma."""
    g = gen(9)
    T, H, D = 3, 2, 64
    dt = torch.float16
    x, dy, w = normal((T, H, D), g, dt), normal((T, H, D), g, dt), normal((D,), g, dt, 0.2, 1.0)
    k = normal((T, 1, D), g, dt)
    pos, f = torch.tensor([0, 7, 90000], dtype=torch.int32, device=DEV), freqs(D)
    dx, _, dw, _ = tcm.qk_norm_rope_bwd(dy, torch.zeros_like(k), x, k, pos, f, w, w, eps=1e-4)
    loss = lambda x, w: (f64(dy) * ol.norm_rope(x, pos.tolist(), f64(f), w, 1e-4)).sum()  # noqa: E731
    r = np.random.default_rng(3)
    h = 1e-5
    for _ in range(8):
        u, z = r.normal(size=(T, H, D)), r.normal(size=D)
        du = (loss(f64(x) + h * u, f64(w)) - loss(f64(x) - h * u, f64(w))) / (2 * h)
        dz = (loss(f64(x), f64(w) + h * z) - loss(f64(x), f64(w) - h * z)) / (2 * h)
        sigma = np.sqrt((ol.half_ulp(f64(dx), "f16") ** 2 / 3).sum())
        assert abs((f64(dx) * u).sum() - du) <= 6 * sigma + 1e-4
        assert abs((f64(dw) * z).sum() - dz) <= 1e-4


def test_backward_same_bits_in_place_and_weight_gradients_alone():
    g = gen(10)
    T, Hq, Hk, D = 1100, 4, 2, 64
    q, k = normal((T, Hq, D), g, torch.bfloat16), normal((T, Hk, D), g, torch.bfloat16)
    gq, gk = normal((T, Hq, D), g, torch.bfloat16), normal((T, Hk, D), g, torch.bfloat16)
    w = normal((D,), g, torch.bfloat16, 0.2, 1.0)
    pos, f = torch.arange(T, dtype=torch.int32, device=DEV), freqs(D)
    one = tcm.qk_norm_rope_bwd(gq, gk, q, k, pos, f, w, w)
    ws = torch.full((tcm.qk_norm_rope_bwd_workspace(D),), 255, dtype=torch.uint8, device=DEV)
    two = tcm.qk_norm_rope_bwd(gq, gk, q, k, pos, f, w, w, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    only = tcm.qk_norm_rope_bwd(gq, gk, q, k, pos, f, None, w)
    assert only[2] is None and torch.equal(only[3], one[3])
    gq2, gk2 = gq.clone(), gk.clone()
    tcm.qk_norm_rope_bwd(gq2, gk2, q, k, pos, f, w, w, dq=gq2, dk=gk2)
    assert torch.equal(gq2, one[0]) and torch.equal(gk2, one[1])
    none = tcm.qk_norm_rope_bwd(gq[:0], gk[:0], q[:0], k[:0], pos[:0], f, w, w)
    assert (none[2] == 0).all() and (none[3] == 0).all()
