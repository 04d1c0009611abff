"""gemm_w4 on the GPU against the float64 oracle.

Tolerance, as the header states it: (K / 32 + 96) 2^-24 of sum |x| scale (q + zero) (E2M1: sum |x w|), and the result's
own rounding.  (A matrix instruction adds 32 products and its operand, at most 33 roundings of the sizes of its own
group; a group has two of them for each 32 values, q's and zero's: 66, and 8 more for the sums they join.  The group's
sum times its scale is rounded once when it is added to those before, K / 32 times at most, whatever waves
share K, and the 16 waves' sums at most 16 times.)
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
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def f64(t):
    return t.double().cpu().numpy()


def make(M, N, K, group=32, elem="u4", zeros=True, dt=BF, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g).to(dt).to(DEV)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).to(DEV)
    if elem == "e2m1":
        return x, w, torch.randint(110, 140, (N, K // 32), generator=g, dtype=torch.uint8).to(DEV), None
    s = (torch.randn((N, K // group), generator=g) * 0.1).to(dt).to(DEV)
    z = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8).to(DEV) if zeros else None
    return x, w, s, z


def check(out, x, w, s, z, elem):
    sc = s.cpu().numpy() if elem == "e2m1" else f64(s)
    ref, mag = os_.gemm_w4(f64(x), w.cpu().numpy(), sc, None if z is None else z.cpu().numpy(), elem)
    u = (x.shape[1] / 32 + 96) * 2.0 ** -24
    tol = u * mag + 1.01 * ol.half_ulp(ref, NAMES[out.dtype])
    got = f64(out)
    if out.dtype is HF:
        # fp16 ends at 65504, and what is half a step (16) or more past it rounds to infinity
        past = np.isinf(got)
        assert (np.sign(ref)[past] == np.sign(got)[past]).all() and (np.abs(ref) + tol >= 65520)[past].all()
        assert past[np.abs(ref) - u * mag >= 65520].all()
        got = np.where(past, ref, got)
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"worst {np.nanmax(err / tol)} at {np.argwhere(~(err <= tol))[:4]}"


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("elem", ["u4", "e2m1"])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 48, 49, 64, 65, 130])
def test_rows(M, elem, dt):
    c = make(M, 80, 416, elem=elem, dt=dt, seed=M)
    check(tcm.gemm_w4(*c, elem=elem), *c, elem)


@pytest.mark.parametrize("elem", ["u4", "e2m1"])
@pytest.mark.parametrize("M", [1, 6, 20, 64])
@pytest.mark.parametrize("N", [1, 7, 15, 16, 17, 31, 33, 63, 65, 129, 1000])
def test_columns(N, M, elem):
    c = make(M, N, 256, elem=elem, dt=HF, seed=N)
    check(tcm.gemm_w4(*c, elem=elem, out_dtype=F32), *c, elem)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("elem", ["u4", "e2m1"])
@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 224, 1024, 1056, 1152, 2016, 4096, 8192])
@pytest.mark.parametrize("M", [1, 40])
def test_depths(M, K, elem, dt):
    c = make(M, 48, K, elem=elem, dt=dt, seed=K)
    check(tcm.gemm_w4(*c, elem=elem), *c, elem)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group,K", [(32, 672), (64, 640), (96, 960), (128, 1024), (128, 384), (160, 800), (256, 2048), (1024, 1024),
                                     (1760, 1760)])
def test_groups(group, K, zeros):
    for M, dt in ((3, BF), (24, HF)):
        c = make(M, 50, K, group, zeros=zeros, dt=dt, seed=group)
        check(tcm.gemm_w4(*c), *c, "u4")


def test_every_element_exactly():
    """x picks one element at a time: every value of q and of a zero point, of E2M1 and of its scale."""
    N, K = 256, 64
    w = torch.randint(0, 256, (N, K // 2), generator=torch.Generator().manual_seed(1), dtype=torch.uint8).to(DEV)
    z = torch.arange(N, dtype=torch.uint8, device=DEV)[:, None].expand(N, 2).contiguous()
    e = torch.arange(N, dtype=torch.uint8, device=DEV)[:, None].expand(N, 2).contiguous()
    for dt in (BF, HF):
        x = torch.eye(K, device=DEV).to(dt)
        out = tcm.gemm_w4(x, w, torch.full((N, 2), 0.5, dtype=dt, device=DEV), z, out_dtype=F32)
        q = torch.tensor(os_.nibbles(w.cpu().numpy()).T.astype(np.float32), device=DEV)
        assert torch.equal(out, (q - z[:, 0].float()) * 0.5)
        out = tcm.gemm_w4(x, w, e, elem="e2m1", out_dtype=F32)
        v = torch.tensor(os_.E2M1[os_.nibbles(w.cpu().numpy())].T, device=DEV) * torch.exp2(e[:, 0].double() - 127)
        # (6 * 2^127 is past fp32)
        assert torch.equal(out[:, :255], v[:, :255].float()) and torch.isnan(out[:, 255]).all()


def test_strides():
    M, N, K = 5, 33, 96
    x, w, s, z = make(M, N, K)
    wide = torch.zeros((M, 2 * K + 8), dtype=BF, device=DEV)
    wide[:, 8:8 + K] = x
    for odt in (BF, F32):
        into = torch.full((M, 3 * N), 5.0, dtype=odt, device=DEV)
        got = tcm.gemm_w4(wide[:, 8:8 + K], w, s, z, out=into[:, N:2 * N])
        assert torch.equal(got, tcm.gemm_w4(x, w, s, z, out_dtype=odt))
        assert (into[:, :N] == 5).all() and (into[:, 2 * N:] == 5).all()


def test_a_row_does_not_reach_another():
    x, w, s, z = make(20, 64, 512, 128)
    clean = tcm.gemm_w4(x, w, s, z)
    x[3, 7], x[17, 500] = float("inf"), float("nan")
    out = tcm.gemm_w4(x, w, s, z)
    keep = [i for i in range(20) if i not in (3, 17)]
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[[3, 17]]).all()
    s2 = s.clone()
    s2[9, 1] = float("nan")
    out = tcm.gemm_w4(x[:2], w, s2, z)
    cols = [i for i in range(64) if i != 9]
    assert torch.isnan(out[:, 9]).all() and torch.equal(out[:, cols], tcm.gemm_w4(x[:2], w, s, z)[:, cols])


def test_nothing_to_do():
    x, w, s, z = make(4, 8, 64)
    assert tcm.gemm_w4(x[:0], w, s, z).shape == (0, 8) and tcm.gemm_w4(x, w[:0], s[:0], z[:0]).shape == (4, 0)
    out = tcm.gemm_w4(x[:, :0], w[:, :0], s[:, :0], None)
    assert (out == 0).all()


def test_large_offsets():
    """Weights past 2^32 bytes (67000 columns of 131072 values): the last columns.  (Groups of 1024 are added 128
    values at a time: K / 128 roundings.)"""
    N, K = 67000, 131072
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device=DEV)
    s = torch.full((N, K // 1024), 0.01, dtype=BF, device=DEV)
    x = torch.randn((2, K), generator=g, device=DEV).to(BF)
    out = tcm.gemm_w4(x, w, s, out_dtype=F32)
    for n in (0, 32768, 65535, 65536, 66999):
        ref, mag = os_.gemm_w4(f64(x), w[n:n + 1].cpu().numpy(), f64(s[n:n + 1]))
        assert (np.abs(f64(out[:, n:n + 1]) - ref) <= (K / 128 + 96) * 2.0 ** -24 * mag).all(), n


# Enough columns that a workgroup takes up to 64 rows, or 32 with X in stages or as a whole
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("M,N,K,group,elem", [
    (33, 16385, 96, 32, "u4"), (48, 16400, 544, 32, "u4"), (49, 16390, 512, 32, "u4"), (63, 16384, 640, 64, "u4"),
    (64, 16417, 1152, 64, "u4"), (40, 16393, 1024, 128, "u4"), (65, 16385, 960, 96, "u4"), (64, 16385, 1280, 256, "u4"),
    (36, 16390, 1056, 32, "e2m1"), (64, 16386, 1152, 32, "e2m1"),
    (17, 2055, 992, 32, "u4"), (32, 2064, 2048, 64, "u4"), (29, 8193, 2304, 64, "u4"), (32, 8200, 2336, 32, "u4"),
    (31, 8197, 2304, 32, "e2m1"), (20, 8196, 2432, 128, "u4"), (15, 2050, 4352, 128, "u4"), (16, 4100, 4384, 32, "e2m1")])
def test_many_columns(M, N, K, group, elem, dt):
    c = make(M, N, K, group, elem=elem, dt=dt, seed=M)
    check(tcm.gemm_w4(*c, elem=elem), *c, elem)


@pytest.mark.parametrize("group,elem", [(32, "u4"), (64, "u4"), (128, "u4"), (32, "e2m1")])
def test_scales_at_any_address(group, elem):
    """Scales and zeros that begin at any element, which decides how many of them a lane loads at once."""
    for M in (3, 20):
        x, w, s, z = make(M, 70, 1024, group, elem=elem, dt=HF, seed=group)
        def moved(t, by):
            room = torch.zeros(t.numel() + 16, dtype=t.dtype, device=DEV)
            at = room[by:by + t.numel()].view(t.shape)
            at.copy_(t)
            return at

        for a, b in ((1, 0), (0, 1), (2, 2), (3, 1), (4, 2), (8, 4)):
            got = tcm.gemm_w4(x, w, moved(s, a), None if z is None else moved(z, b), elem=elem, out_dtype=F32)
            check(got, x, w, s, z, elem)
