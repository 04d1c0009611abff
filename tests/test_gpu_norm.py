"""add_rms_norm, its MXFP8 form and its gradients on the GPU against the float64 oracle.

Tolerances: a lane adds at most 32 squares in a row, 6 steps join a wave and at most 16 waves follow: 54
roundings of the mean, of which the root halves the part; with the sum x + r, 1/D, the root (1 ulp
and a step) and the products 64 roundings, 2^-24 each, cover a value; results are rounded once.  Gradients: as
many of each term's magnitude; weights' sums add one for each row that a workgroup adds and 48 to join.
"""
import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol
from oracle import step as os_

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float32: "f32"}
R = 64 * 2.0 ** -24
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def f64(t):
    return t.double().cpu().numpy()


def rand(shape, seed, dt, sd=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * sd).to(dt).to(DEV)


def within(got, ref, tol, dt):
    err = np.abs(f64(got) - ref)
    tol = tol + 1.01 * ol.half_ulp(ref, NAMES[dt])
    assert (err <= tol).all(), f"worst {np.nanmax(err / tol)} at {np.argwhere(~(err <= tol))[:4]}"


def weight(kind, D, dt):
    return None if kind is None else 1 + rand(D, D, F32, 0.3).to(F32 if kind == "f32" else dt)


def check(x, r, w, y, s, eps=1e-6):
    ref, total = os_.add_rms_norm(f64(x), None if r is None else f64(r), None if w is None else f64(w), eps)
    within(y, ref, R * np.abs(ref) + 1e-37, y.dtype)
    within(s, total, 2.0 ** -23 * np.abs(total), s.dtype)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("D", [8, 16, 504, 512, 520, 2040, 2048, 2056, 4096, 4104, 5120, 8192, 8200, 16384, 32768])
@pytest.mark.parametrize("T", [1, 2, 5, 67])
def test_sizes(T, D, dt):
    kind = [None, "same", "f32"][(T + D // 8) % 3]
    x, r, w = rand((T, D), 1, dt), rand((T, D), 2, dt, 3.0) if T != 2 else None, weight(kind, D, dt)
    out_dtype = F32 if (T + D // 8) % 2 else dt
    y, s = tcm.add_rms_norm(x, w, r, out_dtype=out_dtype)
    assert y.dtype is out_dtype and (s is x) == (r is None)
    check(x, r, w, y, s)


@pytest.mark.parametrize("T", [1000, 2500, 9001])
@pytest.mark.parametrize("D", [64, 1024, 4096])
def test_many_rows(T, D):
    x, r, w = rand((T, D), T, BF), rand((T, D), D, BF), weight("same", D, BF)
    y, s = tcm.add_rms_norm(x, w, r)
    check(x, r, w, y, s)


def test_strides_and_in_place():
    T, D = 9, 264
    wide = rand((T, 3 * D), 5, BF)
    x, r = wide[:, :D], wide[:, 2 * D:]
    keep = wide.clone()
    into = torch.full((T, 2, D), 7.0, dtype=BF, device=DEV)
    y, s = tcm.add_rms_norm(x, None, r, out=into[:, 1], sum_out=wide[:, D:2 * D])
    check(keep[:, :D], keep[:, 2 * D:], None, y, s)
    assert (into[:, 0] == 7).all() and torch.equal(wide[:, :D], keep[:, :D]) and torch.equal(wide[:, 2 * D:], keep[:, 2 * D:])
    for where in ("x", "r"):
        for what in ("sum", "out"):
            a, b = rand((T, D), 6, HF), rand((T, D), 7, HF)
            ref = tcm.add_rms_norm(a, None, b)
            t = a if where == "x" else b
            got = tcm.add_rms_norm(a, None, b, **{"sum_out" if what == "sum" else "out": t})
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_values_that_are_not_finite_stay_in_their_row():
    x = rand((6, 640), 8, BF)
    clean = tcm.add_rms_norm(x)[0]
    x[1, 5], x[3, 600], x[4] = float("inf"), float("nan"), 0.0
    y = tcm.add_rms_norm(x)[0]
    assert torch.equal(y[[0, 2, 5]], clean[[0, 2, 5]]) and (y[4] == 0).all()
    # s / sqrt(inf) is 0 for what is finite, and inf / inf NaN
    assert torch.isnan(y[1, 5]) and (y[1].nan_to_num() == 0).all() and torch.isnan(y[3]).all()
    assert torch.isnan(tcm.add_rms_norm(x[4:5], eps=0.0)[0]).all()


def test_no_rows():
    x = torch.empty((0, 64), dtype=BF, device=DEV)
    assert tcm.add_rms_norm(x, residual=x)[0].shape == (0, 64)
    q, e, _ = tcm.add_rms_norm_mx_fp8(x)
    assert q.shape == (0, 64) and e.shape == (0, 2)
    dx, dw = tcm.add_rms_norm_bwd(x, x, torch.ones(64, dtype=BF, device=DEV))
    assert dx.shape == (0, 64) and (dw == 0).all()


def check_mx(x, r, w, q, e, s):
    ref, total = os_.add_rms_norm(f64(x), None if r is None else f64(r), None if w is None else f64(w))
    T, D = ref.shape
    within(s, total, 2.0 ** -23 * np.abs(total), s.dtype)
    got = e.view(torch.uint8).cpu().numpy().astype(int) - 127
    want = os_.mx_exponents(ref)
    # a largest element within the fp32 error of 448 * 2^e may be on either side
    top = np.abs(ref).reshape(T, -1, 32).max(-1)
    near = np.abs(top / (448 * 2.0 ** np.floor(np.log2(np.maximum(top, 1e-300) / 448) + 0.5)) - 1) < 2 * R
    assert (got == want)[~near].all() and (np.abs(got - want) <= 1).all()
    f = np.repeat(2.0 ** got, 32, 1)
    v = f64(q.view(torch.float8_e4m3fn).float()) * f
    tol = R * np.abs(ref) + 1.01 * ol.half_ulp(ref / f, "e4m3") * f
    assert (np.abs(v - ref) <= tol).all()
    assert (np.abs(v) <= 448 * f).all()


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("T,D", [(1, 32), (3, 96), (1, 4096), (33, 480), (7, 544), (300, 2080), (2, 8224), (5, 32768), (4097, 1024)])
def test_mx(T, D, dt):
    x, r, w = rand((T, D), T, dt), rand((T, D), D, dt, 2.0) if T != 3 else None, weight("f32" if T % 2 else "same", D, dt)
    q, e, s = tcm.add_rms_norm_mx_fp8(x, w, r)
    check_mx(x, r, w, q, e, s)


def test_mx_scales_at_their_borders():
    """Blocks of any size, of zeros, of powers of two and of 448 times them (rows of 64 values whose norm is
    exact: 32 times one magnitude, weights decide), and elements that are not finite."""
    D = 32 * 8
    x = torch.ones((1, D), dtype=BF, device=DEV)
    w = torch.zeros(D, dtype=F32, device=DEV)
    tops = [448.0, 449.0, 2.0 ** -100, 2.0 ** 100, 0.0, 447.0, 1.75, 2.0 ** -126]
    for i, t in enumerate(tops):
        w[32 * i + 3], w[32 * i + 9] = t, -t / 2
    q, e, _ = tcm.add_rms_norm_mx_fp8(x, w, eps=0.0)
    assert (e.view(torch.uint8).int() - 127).tolist() == [[0, 1, -108, 92, -127, 0, -8, -127]]
    v = (q.float() * torch.exp2((e.view(torch.uint8).float() - 127)).repeat_interleave(32, 1))[0]
    for i, t in enumerate(tops):
        if t not in (449.0, 447.0):
            assert v[32 * i + 3] == t and v[32 * i + 9] == -t / 2, t
    w[0], w[1], w[40] = float("inf"), float("nan"), float("-inf")
    q2, e2, _ = tcm.add_rms_norm_mx_fp8(x, w, eps=0.0)
    assert torch.equal(e2, e) and torch.isnan(q2.float()).sum() == 3
    q2.view(torch.uint8)[0, [0, 1, 40]] = q.view(torch.uint8)[0, [0, 1, 40]]
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8))


def test_mx_is_what_the_product_takes():
    T, D, N = 130, 512, 192
    x, r, w = rand((T, D), 1, BF), rand((T, D), 2, BF), weight("same", D, BF)
    q, e, _ = tcm.add_rms_norm_mx_fp8(x, w, r)
    b = rand((N, D), 3, BF).to(torch.float8_e4m3fn).view(torch.uint8)
    sb = torch.full((N, D // 32), 125, dtype=torch.uint8, device=DEV)
    out = tcm.gemm_mx_fp8(q.view(torch.uint8), b, e, sb, out_dtype=F32)
    a = f64(q.float()) * np.repeat(2.0 ** (e.cpu().numpy().astype(float) - 127), 32, 1)
    bb = f64(b.view(torch.float8_e4m3fn).float()) * 0.25
    assert (np.abs(f64(out) - a @ bb.T) <= 1e-4 * (np.abs(a) @ np.abs(bb).T)).all()


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("T,D", [(1, 8), (3, 512), (5, 520), (700, 64), (513, 2048), (1030, 2056), (40, 4096), (2, 8192),
                                 (9, 8200), (3, 32768), (1500, 4096)])
def test_gradients(T, D, dt):
    kind = [None, "same", "f32"][(T + D // 8) % 3]
    s, dy, w = rand((T, D), 1, dt), rand((T, D), 2, dt), weight(kind, D, dt)
    ds = rand((T, D), 3, dt) if T % 2 else None
    dx, dw = tcm.add_rms_norm_bwd(dy, s, w, ds)
    rx, rw, mx, mw = os_.add_rms_norm_bwd(f64(dy), f64(s), None if w is None else f64(w), None if ds is None else f64(ds))
    within(dx, rx, 2 * R * mx, dt)
    if w is None:
        assert dw is None
    else:
        assert (np.abs(f64(dw) - rw) <= (T // 512 + 48 + 64) * 2.0 ** -24 * mw + 1e-30).all()
    again = tcm.add_rms_norm_bwd(dy, s, w, ds)
    assert torch.equal(again[0], dx) and (w is None or torch.equal(again[1], dw))


def test_gradients_in_place_and_strided():
    T, D = 20, 328
    dy, s, ds = (rand((T, D), i, BF) for i in range(3))
    w = weight("same", D, BF)
    ref, rw = tcm.add_rms_norm_bwd(dy, s, w, ds)
    for i in range(3):
        a = [dy.clone(), s.clone(), ds.clone()]
        dx, dw = tcm.add_rms_norm_bwd(a[0], a[1], w, a[2], dx=a[i])
        assert torch.equal(dx, ref) and torch.equal(dw, rw)
    wide = torch.zeros((T, 4, D), dtype=BF, device=DEV)
    for i, t in enumerate((dy, s, ds)):
        wide[:, i] = t
    dx, dw = tcm.add_rms_norm_bwd(wide[:, 0], wide[:, 1], w, wide[:, 2], dx=wide[:, 3],
                                  workspace=torch.empty(tcm.add_rms_norm_bwd_workspace(100, D), dtype=torch.uint8, device=DEV))
    assert torch.equal(dx, ref) and torch.equal(dw, rw) and torch.equal(wide[:, 1], s)


def test_gradients_are_those_of_the_forward_pass():
    """The kernels' forward pass in fp32 results, against differences of it along a direction."""
    T, D = 6, 256
    s, dy = rand((T, D), 1, HF), rand((T, D), 2, HF)
    w = weight("f32", D, HF)
    dx, dw = tcm.add_rms_norm_bwd(dy, s, w)
    u = torch.sign(rand((T, D), 3, HF)) * 2.0 ** -6  # steps that fp16 holds exactly enough
    up, down = (s + u), (s - u)
    f = lambda t: (tcm.add_rms_norm(t, w, out_dtype=F32)[0].double() * dy.double()).sum()  # noqa: E731
    slope = float(f(up) - f(down))
    want = float((dx.double() * (up - down).double()).sum())
    # third-order term: (2^-6)^2 / 6 of slopes of order |dy| / rms each, T * D of them; rounding of dx 2^-12
    scale = float((dy.double().abs() * (up - down).double().abs()).sum())
    assert abs(slope - want) <= (2.0 ** -12 + 2.0 ** -11) * 2 * scale
    v = 2.0 ** -8 * torch.sign(rand(D, 4, F32))
    g = lambda t: (tcm.add_rms_norm(s, t, out_dtype=F32)[0].double() * dy.double()).sum()  # noqa: E731
    up, down = w + v, w - v
    assert abs(float(g(up) - g(down)) - float((dw.double() * (up - down).double()).sum())) <= \
        200 * 2.0 ** -24 * float((dy.double().abs() * 4).sum())
