"""The layer operators' C ABI and binding on the CPU: invalid calls are refused with the
documented status before a device is touched; workspace sizes.  No compute call runs."""
import ctypes

import pytest
import torch

import tensor_core_matrix_amd as tcm

OK, NULLP, BADSHAPE, UNSUP_SHAPE, MISALIGNED, UNSUP_DTYPE, NO_DEVICE, HIP, BADARG, WORKSPACE = range(10)
P = [0x10000 * (i + 1) for i in range(12)]  # 16-byte aligned stand-ins


def _device_visible():
    try:
        return torch.cuda.device_count() > 0
    except Exception:  # pragma: no cover
        return False


# (stand-in addresses must not reach a device)
pytestmark = pytest.mark.skipif(_device_visible(), reason="stand-in pointers must not reach a device")
PASSED = (OK, NO_DEVICE)  # got past validation


def lora(X=P[0], ldx=64, W=P[1], A=P[2], B=P[3], rows=P[4], ranks=None, scales=None, out=P[5], ldo=32, M=4,
         N=32, K=64, L=2, R=16, dt=tcm.BF16, odt=tcm.BF16, ws=P[6], nb=1 << 20):
    return tcm.lib().tcm_lora_gemm_tn(X, ldx, W, A, B, rows, ranks, scales, out, ldo, M, N, K, L, R, dt, odt,
                                      ws, nb, None)


def test_lora_refusals():
    assert lora() in PASSED
    assert lora(odt=tcm.F32) in PASSED and lora(dt=tcm.F16, odt=tcm.F16) in PASSED
    for dt, odt in ((tcm.F32, tcm.F32), (tcm.BF16, tcm.F16), (tcm.F16, tcm.BF16), (tcm.E4M3, tcm.BF16)):
        assert lora(dt=dt, odt=odt) == UNSUP_DTYPE
    for kw in (dict(M=-1), dict(N=-1), dict(K=-8), dict(L=-1), dict(R=-8), dict(ldx=56), dict(ldo=31)):
        assert lora(**kw) == BADSHAPE, kw
    for kw in (dict(R=136), dict(K=(1 << 20) + 8, ldx=(1 << 20) + 8), dict(M=(1 << 30) + 1),
               dict(ldx=(1 << 21) + 8)):
        assert lora(**kw) == UNSUP_SHAPE, kw
    for kw in (dict(X=None), dict(W=None), dict(A=None), dict(B=None), dict(rows=None), dict(out=None),
               dict(ws=None)):
        assert lora(**kw) == NULLP, kw
    for kw in (dict(X=P[0] + 2), dict(W=P[0] + 8), dict(A=P[0] + 4), dict(B=P[0] + 8), dict(out=P[0] + 4),
               dict(ws=P[0] + 8), dict(K=60), dict(ldx=68), dict(R=12)):
        assert lora(**kw) == MISALIGNED, kw
    assert lora(nb=4 * 16 * 4 - 1) == WORKSPACE and lora(nb=4 * 16 * 4) in PASSED


def test_lora_without_adapters_needs_none():
    for kw in (dict(L=0), dict(R=0), dict(K=0, ldx=64)):
        assert lora(A=None, B=None, rows=None, ws=None, nb=0, **kw) in PASSED, kw
    assert lora(X=None, out=None, M=0) == OK and lora(X=None, out=None, N=0) == OK


def test_lora_workspace_covers_every_split():
    for M in (0, 1, 3, 48, 255, 4096):
        for K in (0, 8, 512, 1000, 4096, 1 << 20):
            n = tcm.lora_workspace(M, K, 16)
            assert n % (M * 16 * 4 or 1) == 0 and n <= 8 * M * 16 * 4
            assert n >= M * 16 * 4
    with pytest.raises(tcm.TcmError):
        tcm.lora_workspace(1, 8, 136)
    assert tcm.lib().tcm_lora_workspace(1, 8, 8, None) == NULLP


def heads(ptr=P[0], ts=512, hs=64):
    return tcm.Heads(ptr, ts, hs)


def rope(D=64, rot=64, pos=P[8], freq=P[9], layout=0, norm=1, wq=P[10], wk=P[11], wt=tcm.BF16):
    return tcm.Rope(D, rot, pos, freq, 1.0, layout, norm, 1e-6, wq, wk, wt)


def fwd(q=heads(), k=heads(P[1]), qo=heads(P[2]), ko=heads(P[3]), T=4, Hq=8, Hk=2, r=rope(), dt=tcm.BF16):
    return tcm.lib().tcm_qk_norm_rope(q, k, qo, ko, T, Hq, Hk, r, dt, None)


def test_rope_refusals():
    assert fwd() in PASSED
    assert fwd(r=rope(layout=1, rot=20, D=80), q=heads(ts=640, hs=80), k=heads(ts=640, hs=80),
               qo=heads(ts=640, hs=80), ko=heads(ts=640, hs=80)) in PASSED
    assert fwd(dt=tcm.F32) == UNSUP_DTYPE and fwd(r=rope(wt=tcm.F16)) == UNSUP_DTYPE
    assert fwd(r=rope(wt=tcm.F32)) in PASSED
    assert fwd(r=rope(wt=tcm.F16, wq=None, wk=None)) in PASSED  # no weight, no type
    assert fwd(r=rope(layout=2)) == BADARG and fwd(r=rope(layout=-1)) == BADARG
    assert fwd(T=1 << 30, q=heads(ts=1 << 31)) == BADSHAPE and fwd(q=heads(hs=1 << 60)) == BADSHAPE
    for kw in (dict(T=-1), dict(Hq=-1), dict(Hk=-1), dict(r=rope(D=0, rot=0)), dict(r=rope(rot=72)),
               dict(r=rope(rot=31)), dict(r=rope(rot=-2)), dict(q=heads(ts=-512)), dict(qo=heads(ts=256)),
               dict(ko=heads(hs=32)), dict(qo=heads(hs=0))):
        assert fwd(**kw) == BADSHAPE, kw
    for kw in (dict(r=rope(D=264, rot=0)), dict(r=rope(D=68, rot=0)), dict(T=(1 << 30) + 1), dict(Hq=65536)):
        assert fwd(**kw) == UNSUP_SHAPE, kw
    for kw in (dict(q=None), dict(ko=None), dict(q=heads(None)), dict(r=None), dict(r=rope(pos=None)),
               dict(r=rope(freq=None))):
        assert fwd(**kw) == NULLP, kw
    assert fwd(r=rope(rot=0, pos=None, freq=None)) in PASSED
    for kw in (dict(q=heads(P[0] + 8)), dict(k=heads(ts=516)), dict(qo=heads(hs=68)), dict(r=rope(wq=P[10] + 2)),
               dict(r=rope(wk=P[10] + 8))):
        assert fwd(**kw) == MISALIGNED, kw
    assert fwd(T=0, q=None, k=None, qo=None, ko=None) == OK
    assert fwd(Hq=0, q=None, qo=None) in PASSED and fwd(Hk=0, k=None, ko=None) in PASSED
    # heads outside, tokens inside is a view as well
    assert fwd(qo=heads(ts=64, hs=256)) in PASSED and fwd(qo=heads(ts=64, hs=192)) == BADSHAPE


def cache(k=P[4], v=P[5], pages=3, page_size=16, ks=(2048, 128, 64), vs=(2048, 128, 64), dt=tcm.BF16):
    return tcm.Cache(k, v, pages, page_size, *ks, *vs, dt, 1.0, 1.0)


def into(c=cache(), slots=P[6], v=heads(P[7]), T=4, Hk=2, r=rope(), dt=tcm.BF16):
    return tcm.lib().tcm_qk_norm_rope_cache(heads(), heads(P[1]), v, heads(P[2]), c, slots, T, 8, Hk, r, dt, None)


def test_rope_cache_refusals():
    assert into() in PASSED and into(cache(dt=tcm.E4M3)) in PASSED
    assert into(cache(k=None, v=None, pages=0)) in PASSED
    assert into(cache(dt=tcm.F16)) == UNSUP_DTYPE and into(cache(dt=tcm.F32)) == UNSUP_DTYPE
    for c in (cache(pages=-1), cache(page_size=0), cache(ks=(2048, 128, -64)), cache(ks=(2048, 128, 32)),
              cache(vs=(2048, 8, 64)), cache(vs=(1 << 41, 128, 64)),
              cache(pages=1 << 30, ks=(1 << 40, 128, 64))):
        assert into(c) == BADSHAPE
    assert into(cache(page_size=(1 << 20) + 1)) == UNSUP_SHAPE
    for kw in (dict(c=None), dict(c=cache(k=None)), dict(c=cache(v=None)), dict(slots=None), dict(v=None)):
        assert into(**kw) == NULLP, kw
    for c in (cache(k=P[4] + 8), cache(ks=(2048, 132, 64)), cache(dt=tcm.E4M3, vs=(2048, 136, 64))):
        assert into(c) == MISALIGNED
    assert into(T=0, slots=None, v=None) == OK


def bwd(dqo=heads(), dko=heads(P[1]), q=heads(P[2]), k=heads(P[3]), dq=heads(P[4]), dk=heads(P[5]), wq=P[6],
        wk=P[7], T=4, r=rope(), dt=tcm.BF16, ws=P[8], nb=1 << 20):
    return tcm.lib().tcm_qk_norm_rope_bwd(dqo, dko, q, k, dq, dk, wq, wk, T, 8, 2, r, dt, ws, nb, None)


def test_rope_bwd_refusals():
    need = tcm.qk_norm_rope_bwd_workspace(64)
    assert bwd() in PASSED and bwd(nb=need) in PASSED and bwd(nb=need - 1) == WORKSPACE
    assert bwd(wq=None, wk=None, ws=None, nb=0) in PASSED
    assert bwd(ws=None) == NULLP and bwd(ws=P[8] + 8) == MISALIGNED
    bare = rope(norm=0, wq=None, wk=None)
    assert bwd(r=bare) == BADARG  # weight gradients of no norm
    assert bwd(r=bare, wq=None, wk=None, q=None, k=None) in PASSED
    for kw in (dict(dqo=None), dict(dko=None), dict(q=None), dict(k=None), dict(dq=None), dict(dk=None)):
        assert bwd(**kw) == NULLP, kw
    assert bwd(dq=heads(P[4], ts=256)) == BADSHAPE and bwd(dko=heads(P[1] + 2)) == MISALIGNED
    assert bwd(dt=tcm.F32) == UNSUP_DTYPE
    assert bwd(T=0, wq=None, wk=None, dqo=None, dko=None) == OK
    for D in (0, -8):
        with pytest.raises(tcm.TcmError):
            tcm.qk_norm_rope_bwd_workspace(D)


def attn(q=heads(), c=cache(), table=P[6], ts=8, lengths=P[7], most=128, out=heads(P[2]), lse=None, B=4, Hq=8,
         Hk=2, D=64, window=0, dt=tcm.BF16, ws=None, nb=0):
    return tcm.lib().tcm_paged_attention(q, c, table, ts, lengths, most, out, lse, B, Hq, Hk, D, 1.0, window, dt,
                                         ws, nb, None)


def test_attention_refusals():
    assert attn() in PASSED and attn(window=5, lse=P[9]) in PASSED
    assert attn(c=cache(dt=tcm.E4M3)) in PASSED
    assert attn(dt=tcm.F32) == UNSUP_DTYPE and attn(c=cache(dt=tcm.F16)) == UNSUP_DTYPE
    for kw in (dict(B=-1), dict(Hq=-8), dict(Hq=7), dict(Hk=0), dict(Hk=3), dict(D=0), dict(most=-1),
               dict(window=-1), dict(ts=-1), dict(out=heads(ts=64)), dict(c=cache(ks=(2048, -8, 64)))):
        assert attn(**kw) == BADSHAPE, kw
    assert attn(B=65535, Hq=65535, Hk=65535, q=heads(ts=65535 * 64), out=heads(ts=65535 * 64)) == UNSUP_SHAPE
    for kw in (dict(B=65536), dict(D=264), dict(D=60), dict(most=(1 << 30) + 1), dict(ts=1 << 31)):
        assert attn(**kw) == UNSUP_SHAPE, kw
    for kw in (dict(q=None), dict(c=None), dict(c=cache(k=None)), dict(table=None), dict(lengths=None),
               dict(out=None)):
        assert attn(**kw) == NULLP, kw
    assert attn(table=None, ts=0) in PASSED  # no room for a key
    assert attn(c=cache(k=None, v=None, pages=0)) in PASSED
    for kw in (dict(q=heads(P[0] + 8)), dict(c=cache(v=P[5] + 8)), dict(c=cache(vs=(2048, 132, 64))),
               dict(D=72, c=cache(dt=tcm.E4M3, ks=(2304, 144, 80), vs=(2304, 144, 80)))):
        assert attn(**kw) == MISALIGNED, kw
    assert attn(B=0, q=None, out=None, lengths=None) == OK


def test_attention_workspace():
    """One sequence of many keys is split and needs one; the size covers every shorter
    call and every window."""
    need = tcm.paged_attention_workspace(1, 8, 2, 64, 1 << 16)
    assert need > 0
    big = dict(B=1, most=1 << 16, ts=1 << 12)
    assert attn(**big) == NULLP and attn(**big, ws=P[9], nb=64) == WORKSPACE
    assert attn(**big, ws=P[9] + 8, nb=need) == MISALIGNED
    for most in (0, 1, 255, 256, 257, 25600, 25601, 40000, 65535, 1 << 16):
        for window in (0, 1, 300, 25600):
            assert attn(B=1, most=most, ts=1 << 12, window=window, ws=P[9], nb=need) in PASSED
    assert tcm.paged_attention_workspace(0, 8, 2, 64, 100) == 0
    assert tcm.lib().tcm_paged_attention_workspace(1, 8, 2, 64, 10, None) == NULLP


# ---- the binding: wrong tensors are refused before the library is called ------------------

def test_binding_refuses_wrong_tensors():
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)  # noqa: E731
    x, w, a, b, rows = z(4, 64), z(32, 64), z(2, 16, 64), z(2, 32, 16), z(4, dt=i32)
    with pytest.raises(ValueError):
        tcm.lora_gemm_tn(x, w, a, b, rows)  # on the CPU
    for bad, err in (((x.float(), w, a, b, rows), TypeError), ((x, w.half(), a, b, rows), TypeError),
                     ((x, w[:, :32], a, b, rows), ValueError), ((x, w, a, b[:, :, :8], rows), ValueError),
                     ((x, w, a, b, rows.long()), TypeError), ((x, w, a, b, rows[:3]), ValueError),
                     ((x.t().contiguous().t(), w, a, b, rows), ValueError)):
        with pytest.raises(err):
            tcm.lora_gemm_tn(*bad)
    with pytest.raises(TypeError):
        tcm.lora_gemm_tn(x, w, a, b, rows, scales=z(2))
    with pytest.raises(TypeError):
        tcm.lora_gemm_tn(x, w, a, b, rows, out_dtype=torch.float16)
    q, k, pos, f = z(4, 8, 64), z(4, 2, 64), z(4, dt=i32), z(32, dt=torch.float64)
    with pytest.raises(ValueError):
        tcm.qk_norm_rope(q, k, pos, f)  # on the CPU
    for kw, err in ((dict(positions=pos.long()), TypeError), (dict(positions=pos[:2]), ValueError),
                    (dict(inv_freq=f.float()), TypeError), (dict(layout="other"), ValueError),
                    (dict(wq=z(63)), ValueError), (dict(wq=z(64, dt=torch.float16)), TypeError),
                    (dict(wq=z(64), norm=False), ValueError), (dict(q_out=z(4, 8, 64, dt=f32)), TypeError),
                    (dict(k_out=z(4, 8, 64)), ValueError), (dict(wq=z(64), wk=z(64, dt=f32)), TypeError)):
        with pytest.raises(err):
            tcm.qk_norm_rope(q, k, **{**dict(positions=pos, inv_freq=f), **kw})
    kc, table, n = z(3, 16, 2, 64), z(4, 2, dt=i32), z(4, dt=i32)
    with pytest.raises(ValueError):
        tcm.paged_attention(q, kc, kc, table, n)  # on the CPU
    for bad, err in (((q.float(), kc, kc, table, n), TypeError), ((q, kc, kc.half(), table, n), ValueError),
                     ((q, kc.half(), kc.half(), table, n), TypeError), ((q, kc, kc, table.long(), n), ValueError),
                     ((q, kc, kc, table, n[:2]), ValueError), ((q, kc, kc, table[:2], n), ValueError),
                     ((q, kc[..., :32], kc[..., :32], table, n), ValueError)):
        with pytest.raises(err):
            tcm.paged_attention(*bad)


def test_structures_match_the_header():
    """Sizes and offsets of the structures as a C compiler lays them out."""
    import os
    import subprocess
    import tempfile

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    structs = {"tcm_heads": tcm.Heads, "tcm_cache": tcm.Cache, "tcm_rope": tcm.Rope}
    lines = []
    for name, t in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in t._fields_]
    src = '#include <stddef.h>\n#include <stdio.h>\n#include "tcm.h"\nint main(void) {' + "".join(lines) + "return 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        with open(os.path.join(d, "s.c"), "w") as fh:
            fh.write(src)
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), os.path.join(d, "s.c"), "-o",
                        os.path.join(d, "s")], check=True)
        got = [int(x) for x in subprocess.run([os.path.join(d, "s")], capture_output=True, check=True).stdout.split()]
    want = []
    for t in structs.values():
        want.append(ctypes.sizeof(t))
        want += [getattr(t, f).offset for f, _ in t._fields_]
    assert got == want
