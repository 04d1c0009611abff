"""The C ABI and binding of a drafting step's operators on the CPU: invalid calls are refused with the
documented status before a device is touched; workspace sizes.  No compute call runs."""
import pytest
import torch

import tensor_core_matrix_amd as tcm
from test_layer_abi import (BADARG, BADSHAPE, MISALIGNED, NULLP, OK, P, PASSED, UNSUP_DTYPE, UNSUP_SHAPE, WORKSPACE,
                            _device_visible, cache, heads)

# (stand-in addresses must not reach a device)
pytestmark = pytest.mark.skipif(_device_visible(), reason="stand-in pointers must not reach a device")


def plan(lengths=P[0], change=P[1], table=P[2], ts=16, per=16, B=4, pages=64, page=16, stack=P[3], cap=64, count=P[4],
         starts=P[5], slots=P[6], positions=P[7], T=32, missing=P[8]):
    return tcm.lib().tcm_cache_plan(lengths, change, table, ts, per, B, pages, page, stack, cap, count, starts, slots,
                                    positions, T, missing, None)


def test_plan_refusals():
    assert plan() in PASSED and plan(slots=None, positions=None, missing=None) in PASSED
    assert plan(B=0, lengths=None, change=None, table=None) in PASSED and plan(cap=0, stack=None) in PASSED
    for kw in (dict(B=-1), dict(per=-1), dict(ts=15), dict(pages=-1), dict(page=0), dict(cap=-1), dict(T=-1)):
        assert plan(**kw) == BADSHAPE, kw
    for kw in (dict(B=65536), dict(page=(1 << 20) + 1, pages=0, per=0), dict(pages=1 << 27), dict(per=1 << 27, ts=1 << 27),
               dict(T=(1 << 30) + 1), dict(cap=1 << 31), dict(ts=1 << 31)):
        assert plan(**kw) == UNSUP_SHAPE, kw
    for kw in (dict(lengths=None), dict(change=None), dict(table=None), dict(stack=None), dict(count=None),
               dict(starts=None)):
        assert plan(**kw) == NULLP, kw
    assert plan(B=1, ts=0) in PASSED  # no step from row to row


def norm(X=P[0], ldx=64, r=P[1], ldr=64, w=P[2], wt=tcm.BF16, s=P[3], lds=64, out=P[4], ldo=64, T=4, D=64, dt=tcm.BF16,
         odt=tcm.BF16):
    return tcm.lib().tcm_add_rms_norm(X, ldx, r, ldr, w, wt, 1e-6, s, lds, out, ldo, T, D, dt, odt, None)


def mx(X=P[0], ldx=64, r=P[1], ldr=64, w=P[2], wt=tcm.BF16, s=P[3], lds=64, out=P[4], scale=P[5] + 1, T=4, D=64,
       dt=tcm.BF16):
    return tcm.lib().tcm_add_rms_norm_mx_fp8(X, ldx, r, ldr, w, wt, 1e-6, s, lds, out, scale, T, D, dt, None)


def bwd(dy=P[0], lddy=64, ds=P[1], ldds=64, s=P[2], lds=64, w=P[3], wt=tcm.BF16, dx=P[4], lddx=64, dw=P[5], T=4, D=64,
        dt=tcm.BF16, ws=P[6], nb=4 * 64 * 4):
    return tcm.lib().tcm_add_rms_norm_bwd(dy, lddy, ds, ldds, s, lds, w, wt, 1e-6, dx, lddx, dw, T, D, dt, ws, nb, None)


def test_norm_refusals():
    assert norm() in PASSED and norm(odt=tcm.F32) in PASSED and norm(dt=tcm.F16, odt=tcm.F16, wt=tcm.F32) in PASSED
    assert norm(r=None, w=None, s=None, ldr=0, lds=0, wt=tcm.E4M3) in PASSED and norm(T=1, ldx=0, ldr=3, lds=-1, ldo=7) in PASSED
    assert norm(T=0, X=None, out=None) == OK and mx() in PASSED and mx(T=0, X=None) == OK
    for kw in (dict(dt=tcm.F32, odt=tcm.F32), dict(odt=tcm.F16), dict(wt=tcm.F16), dict(odt=tcm.E4M3)):
        assert norm(**kw) == UNSUP_DTYPE, kw
    assert mx(dt=tcm.E4M3) == UNSUP_DTYPE and mx(wt=tcm.F16) == UNSUP_DTYPE
    for kw in (dict(T=-1), dict(D=0), dict(ldx=63), dict(ldr=56), dict(lds=63), dict(ldo=63), dict(ldx=1 << 62)):
        assert norm(**kw) == BADSHAPE, kw
    for kw in (dict(T=(1 << 30) + 1), dict(D=32776, ldx=32776, ldr=32776, lds=32776, ldo=32776)):
        assert norm(**kw) == UNSUP_SHAPE, kw
    for kw in (dict(X=None), dict(out=None)):
        assert norm(**kw) == NULLP, kw
    assert mx(out=None) == NULLP and mx(scale=None) == NULLP
    for kw in (dict(X=P[0] + 2), dict(r=P[0] + 8), dict(w=P[0] + 4), dict(s=P[0] + 8), dict(out=P[0] + 8), dict(ldx=68),
               dict(ldr=68), dict(lds=68), dict(ldo=68), dict(D=60)):
        assert norm(**kw) == MISALIGNED, kw
    assert norm(odt=tcm.F32, ldo=68) in PASSED and norm(odt=tcm.F32, ldo=66) == MISALIGNED
    assert mx(D=40) == MISALIGNED and mx(out=P[0] + 8) == MISALIGNED


def test_norm_backward_refusals():
    assert bwd() in PASSED and bwd(ds=None, w=None, dw=None, ws=None, nb=0) in PASSED
    assert bwd(T=0, dy=None, s=None, dx=None, dw=None) == OK and bwd(T=0, dy=None, s=None, dx=None, ws=None, nb=0) in PASSED
    for kw in (dict(dy=None), dict(s=None), dict(dx=None), dict(ws=None)):
        assert bwd(**kw) == NULLP, kw
    for kw in (dict(lddy=56), dict(ldds=56), dict(lds=56), dict(lddx=56), dict(T=-1), dict(D=0)):
        assert bwd(**kw) == BADSHAPE, kw
    for kw in (dict(dy=P[0] + 2), dict(ds=P[0] + 2), dict(s=P[0] + 2), dict(dx=P[0] + 2), dict(w=P[0] + 2),
               dict(ws=P[0] + 4), dict(D=60)):
        assert bwd(**kw) == MISALIGNED, kw
    assert bwd(nb=4 * 64 * 4 - 1) == WORKSPACE and bwd(dt=tcm.F32) == UNSUP_DTYPE and bwd(wt=tcm.F16) == UNSUP_DTYPE
    last = 0
    for T in (0, 1, 3, 511, 512, 513, 100000, 1 << 30):  # enough also for fewer rows
        n = tcm.add_rms_norm_bwd_workspace(T, 64)
        assert last <= n and bwd(T=T, nb=n) in PASSED
        last = n
    with pytest.raises(tcm.TcmError):
        tcm.add_rms_norm_bwd_workspace(4, 40000)


def w4(X=P[0], ldx=64, W=P[1], s=P[2], z=P[3], out=P[4], ldo=32, M=4, N=32, K=64, group=32, elem=tcm.U4, dt=tcm.BF16,
       odt=tcm.BF16):
    return tcm.lib().tcm_gemm_w4(X, ldx, W, s, z, out, ldo, M, N, K, group, elem, dt, odt, None)


def test_w4_refusals():
    assert w4() in PASSED and w4(z=None, odt=tcm.F32) in PASSED and w4(group=64, dt=tcm.F16, odt=tcm.F16) in PASSED
    assert w4(elem=tcm.E2M1, z=None, s=P[2] + 1) in PASSED and w4(M=1, ldx=3, ldo=-1) in PASSED
    assert w4(M=0, X=None) == OK and w4(N=0, out=None) == OK and w4(K=0, X=None, W=None, s=None, z=None) in PASSED
    for kw in (dict(dt=tcm.F32, odt=tcm.F32), dict(odt=tcm.F16), dict(elem=tcm.E4M3), dict(elem=99)):
        assert w4(**kw) == UNSUP_DTYPE, kw
    for kw in (dict(M=-1), dict(N=-1), dict(K=-32), dict(group=0), dict(ldx=56), dict(ldo=31)):
        assert w4(**kw) == BADSHAPE, kw
    for kw in (dict(K=48), dict(group=48), dict(K=96, ldx=96, group=64), dict(group=64, elem=tcm.E2M1, z=None),
               dict(K=(1 << 20) + 32, ldx=(1 << 20) + 32), dict(M=(1 << 30) + 1), dict(N=(1 << 30) + 1, ldo=(1 << 30) + 1),
               dict(ldx=(1 << 21) + 8), dict(ldo=1 << 31), dict(M=64 * 65536)):
        assert w4(**kw) == UNSUP_SHAPE, kw
    for kw in (dict(X=None), dict(W=None), dict(s=None), dict(out=None)):
        assert w4(**kw) == NULLP, kw
    assert w4(elem=tcm.E2M1) == BADARG  # zero points
    for kw in (dict(X=P[0] + 8), dict(W=P[0] + 8), dict(s=P[0] + 1), dict(out=P[0] + 1), dict(out=P[0] + 2, odt=tcm.F32),
               dict(ldx=68)):
        assert w4(**kw) == MISALIGNED, kw


def tree(q=None, c=None, table=P[3], ts=64, lengths=P[4], most=1024, starts=P[5], nodes=8, bits=P[6], words=1, out=None,
         lse=P[8], T=16, B=2, Hq=8, Hk=2, D=64, window=0, dt=tcm.BF16, ws=P[9], nb=1 << 40):
    return tcm.lib().tcm_paged_tree_attention(q or heads(), c or cache(), table, ts, lengths, most, starts, nodes, bits,
                                              words, out or heads(P[7]), lse, T, B, Hq, Hk, D, 0.125, window, dt, ws, nb,
                                              None)


def test_tree_refusals():
    assert tree() in PASSED and tree(bits=None, words=0, lse=None) in PASSED and tree(c=cache(dt=tcm.E4M3)) in PASSED
    for kw in (dict(T=0), dict(B=0), dict(nodes=0), dict(Hq=0, Hk=0)):
        assert tree(lengths=None, starts=None, **kw) == OK, kw
    for kw in (dict(T=-1), dict(B=-1), dict(nodes=-1), dict(most=-1), dict(window=-1), dict(ts=-1), dict(words=-1),
               dict(nodes=65), dict(Hq=7), dict(Hk=0), dict(D=0), dict(out=heads(P[7], hs=56))):
        assert tree(**kw) == BADSHAPE, kw
    for kw in (dict(B=65536), dict(Hq=65536, Hk=1), dict(D=264), dict(D=60), dict(most=(1 << 30) + 1), dict(T=(1 << 30) + 1),
               dict(nodes=1 << 29, words=1 << 23), dict(ts=1 << 31), dict(words=1 << 30)):
        assert tree(**kw) == UNSUP_SHAPE, kw
    for kw in (dict(lengths=None), dict(starts=None), dict(table=None), dict(q=heads(None)), dict(out=heads(None)),
               dict(ws=None)):
        assert tree(**kw) == NULLP, kw
    for kw in (dict(bits=P[6] + 4), dict(q=heads(P[0] + 2)), dict(out=heads(P[7] + 8)), dict(ws=P[9] + 8),
               dict(D=72, c=cache(dt=tcm.E4M3))):
        assert tree(**kw) == MISALIGNED, kw
    for kw in (dict(dt=tcm.F32), dict(c=cache(dt=tcm.F16))):
        assert tree(**kw) == UNSUP_DTYPE, kw
    need = tcm.paged_tree_attention_workspace(2, 8, 2, 64, 8, 1024)
    assert tree(nb=need - 1) == WORKSPACE and tree(nb=need) in PASSED and tree(nb=0, ws=None, most=64) in PASSED


def test_tree_workspaces_cover_smaller_calls():
    """The size for given most is enough for every smaller number of sequences, tokens and keys, and every window."""
    for Hq, Hk in ((8, 2), (4, 4), (64, 1)):
        for D in (64, 256):
            for B, nodes, most in ((1, 1, 300), (3, 9, 5000), (40, 64, 4096), (200, 5, 70000), (5000, 2, 1000)):
                n = tcm.paged_tree_attention_workspace(B, Hq, Hk, D, nodes, most)
                for b in {x for x in (1, 2, B // 3, B - 1, B) if 0 < x <= B}:
                    for x in {1, nodes // 2, nodes - 1, nodes} - {0}:
                        for y in {0, 1, 255, 256, 257, most // 3, most}:
                            for w in (0, 1, 200):
                                assert tree(B=b, nodes=x, most=y, Hq=Hq, Hk=Hk, D=D, window=w, nb=n, T=10 ** 6,
                                            q=heads(ts=Hq * D, hs=D), out=heads(P[7], ts=Hq * D, hs=D),
                                            c=cache(ks=(16 * Hk * D, Hk * D, D), vs=(16 * Hk * D, Hk * D, D))) in PASSED, \
                                    (Hq, Hk, D, B, nodes, most, b, x, y, w)


def test_binding_refusals():
    bf, i32 = torch.bfloat16, torch.int32
    x = torch.zeros((4, 64), dtype=bf)
    t = torch.zeros
    for f, e in ((lambda: tcm.add_rms_norm(x.float()), TypeError), (lambda: tcm.add_rms_norm(x, t(64)), ValueError),
                 (lambda: tcm.add_rms_norm(x, t(32, dtype=bf)), ValueError), (lambda: tcm.add_rms_norm(x, t(64, dtype=torch.float16)), TypeError),
                 (lambda: tcm.add_rms_norm(x, residual=x[:2]), ValueError), (lambda: tcm.add_rms_norm(x, residual=x.half()), TypeError),
                 (lambda: tcm.add_rms_norm(x.t()), ValueError), (lambda: tcm.add_rms_norm(x, out=t((4, 64), dtype=torch.half)), TypeError),
                 (lambda: tcm.add_rms_norm_mx_fp8(x, scale=t((4, 3), dtype=torch.uint8)), ValueError),
                 (lambda: tcm.add_rms_norm_mx_fp8(x, out=x), TypeError), (lambda: tcm.add_rms_norm_bwd(x, x.half()), TypeError),
                 (lambda: tcm.gemm_w4(x, t((8, 32), dtype=torch.uint8), t((8, 2), dtype=bf), elem="u8"), ValueError),
                 (lambda: tcm.gemm_w4(x, t((8, 32), dtype=torch.uint8), t((8, 2))), TypeError),
                 (lambda: tcm.gemm_w4(x, t((8, 32), dtype=torch.uint8), t((8, 3), dtype=bf)), ValueError),
                 (lambda: tcm.gemm_w4(x, t((8, 32), dtype=i32), t((8, 2), dtype=bf)), TypeError),
                 (lambda: tcm.gemm_w4(x, t((8, 32), dtype=torch.uint8), t((8, 2), dtype=bf), t((8, 2), dtype=i32)), TypeError),
                 (lambda: tcm.gemm_w4(x, t((8, 32), dtype=torch.uint8), t((8, 2), dtype=bf), elem="e2m1"), TypeError),
                 (lambda: tcm.cache_plan(t(4, dtype=i32), t(3, dtype=i32), t((4, 2), dtype=i32), t(8, dtype=i32),
                                         t(1, dtype=i32), 16, 8), ValueError),
                 (lambda: tcm.cache_plan(t(4, dtype=i32), t(4, dtype=i32), t((4, 2), dtype=i32), t(8, dtype=i32),
                                         t(1, dtype=i32), 16), ValueError),
                 (lambda: tcm.cache_plan(t(4, dtype=i32), t(4), t((4, 2), dtype=i32), t(8, dtype=i32), t(1, dtype=i32), 16, 8), TypeError)):
        with pytest.raises(e):
            f()
    # all in order, but not on a GPU
    with pytest.raises(ValueError, match="GPU"):
        tcm.add_rms_norm(x)
    with pytest.raises(ValueError, match="GPU"):
        tcm.gemm_w4(x, t((8, 32), dtype=torch.uint8), t((8, 2), dtype=bf))
    q, kc, i = t((6, 8, 64), dtype=bf), t((4, 16, 2, 64), dtype=bf), lambda *s: t(s, dtype=i32)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        tcm.paged_tree_attention(q, kc, kc, i(2, 2), i(2), i(3), 3)
    for kw, e in ((dict(tree=t(6, dtype=torch.int64)), ValueError), (dict(tree=t((6, 1), dtype=i32)), TypeError),
                  (dict(tree=t((5, 1), dtype=torch.int64)), ValueError)):
        with pytest.raises(e):
            tcm.paged_tree_attention(q, kc, kc, i(2, 2), i(2), i(3), 3, **kw)
    with pytest.raises(ValueError):
        tcm.paged_tree_attention(q, kc, kc, i(2, 2), i(2), i(2), 3)
