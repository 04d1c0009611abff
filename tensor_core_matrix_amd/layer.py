"""The layer around the products: a projection with low-rank adapters, the norm and
rotation of query and key heads, a paged key-value cache and the attention of one
new token over it (C ABI in ``include/tcm.h``).

As in the rest of the binding, a call only marshals tensors into pointers, sizes,
strides and the current stream of their device.  All tensors of a call lie on one
device; index tensors are int32.  A ``workspace`` is a uint8 tensor of at least the
bytes the matching ``*_workspace`` function gives, of any contents; without one the
call takes one from torch's allocator, on the current stream.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import BF16, E4M3, F16, F32, Cache, Heads, Rope, _check, lib

__all__ = ["lora_gemm_tn", "lora_workspace", "qk_norm_rope", "qk_norm_rope_cache",
           "qk_norm_rope_bwd", "qk_norm_rope_bwd_workspace", "paged_attention",
           "paged_attention_workspace", "rope_frequencies"]

_HALF = {torch.float16: F16, torch.bfloat16: BF16}
_OUT = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
_LAYOUTS = {"half": 0, "interleaved": 1}


# The current stream's handle without making a Stream object (2 us a call, a third of a
# small call's whole time on the host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _half(t, what):
    code = _HALF.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float16 or bfloat16, not {t.dtype}")
    return code


def _expect(t, what, shape, dtype, dev):
    """t as a dense tensor of this shape, type and device (index): its address."""
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous and on the first tensor's device")
    return t.data_ptr()


def _heads(t, what, shape, dtype, dev):
    """The view (tokens, heads, D) of t; the elements of a head must be contiguous."""
    ts, hs, ds = t.stride() if t.dim() == 3 else (0, 0, 0)
    if t.dtype is dtype and t.shape == shape and ds == 1 and t.get_device() == dev:
        return Heads(t.data_ptr(), ts, hs)
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {shape}, not {tuple(t.shape)}")
    raise ValueError(f"{what} must have contiguous heads and be on the first tensor's device")


def _cache(k, v, k_scale, v_scale, Hk, D, dtype, dev):
    shape = k.shape
    if k.dtype is not v.dtype or shape != v.shape or len(shape) != 4 or shape[2] != Hk or shape[3] != D:
        raise ValueError(f"k_cache and v_cache must be (pages, page_size, {Hk}, {D}) of one type")
    if k.dtype is dtype:
        code = _HALF[dtype]
    elif k.dtype in (torch.float8_e4m3fn, torch.uint8):
        code = E4M3
    else:
        raise TypeError(f"a cache is {dtype}, float8_e4m3fn or uint8 (E4M3 bytes), not {k.dtype}")
    kp, kt, kh, ke = k.stride()
    vp, vt, vh, ve = v.stride()
    if ke != 1 or ve != 1 or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("caches must have contiguous heads and be on the first tensor's device")
    return Cache(k.data_ptr(), v.data_ptr(), shape[0], shape[1], kp, kt, kh, vp, vt, vh, code, k_scale,
                 v_scale)


def _rope(T, D, positions, inv_freq, wq, wk, eps, layout, factor, norm, dtype, dev):
    rot = 2 * inv_freq.shape[0] if inv_freq is not None else 0
    pos = freq = a = b = None
    if rot:
        pos = _expect(positions, "positions", (T,), torch.int32, dev)
        freq = _expect(inv_freq, "inv_freq", (rot // 2,), torch.float64, dev)
    kind = _LAYOUTS.get(layout)
    if kind is None:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, not {layout!r}")
    wt = wk.dtype if wk is not None else wq.dtype if wq is not None else dtype
    if not norm and (wq is not None or wk is not None):
        raise ValueError("weights belong to the norm: norm=False takes none")
    if wt is not dtype and wt is not torch.float32:
        raise TypeError(f"weights must be {dtype} or float32, not {wt}")
    if wq is not None:
        a = _expect(wq, "wq", (D,), wt, dev)
    if wk is not None:
        b = _expect(wk, "wk", (D,), wt, dev)
    return Rope(D, rot, pos, freq, factor, kind, 1 if norm else 0, eps, a, b, _OUT[wt])


def _bytes(f, *sizes):
    n = ctypes.c_int64()
    _check(f(*sizes, ctypes.byref(n)))
    return n.value


def _workspace(ws, dev, size, *sizes):
    """(pointer, bytes, the tensor) of the given workspace, or of a new one of
    size(*sizes) bytes."""
    if dev < 0:
        raise ValueError("tensors must be on a GPU")
    if ws is None:
        need = size(*sizes)
        if need == 0:
            return None, 0, None
        ws = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", dev))
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("workspace must be contiguous and on the first tensor's device")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def _run(dev, f, *args):
    """f(*args, stream) on the device's current stream."""
    if dev < 0:
        raise ValueError("tensors must be on a GPU")
    if dev == torch.cuda.current_device():
        status = f(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _raw_stream(dev))
    if status:
        _check(status)


def lora_workspace(M, K, R):
    """Bytes of workspace of lora_gemm_tn, enough also for fewer rows, a smaller K or R."""
    return _bytes(lib().tcm_lora_workspace, M, K, R)


def lora_gemm_tn(x, w, lora_a, lora_b, row_adapter, scales=None, ranks=None, out=None,
                 out_dtype=None, workspace=None):
    """out[i] = x[i] . w^T + scales[a] (x[i] . lora_a[a]^T) . lora_b[a]^T with
    a = row_adapter[i] (outside 0 .. L-1, -1 by custom: the first term alone).
    x (M, K) with contiguous rows, w (N, K), lora_a (L, R, K), lora_b (L, N, R)
    float16/bfloat16; row_adapter (M,) int32; scales (L,) float32; ranks (L,)
    int32: only the first ranks[a] rows of lora_a[a] and columns of lora_b[a]
    are used; out (M, N) of x's type or float32, with contiguous rows."""
    code = _half(x, "x")
    dev = x.get_device()
    M, K = x.shape
    N = w.shape[0]
    L, R = lora_a.shape[:2]
    wp = _expect(w, "w", (N, K), x.dtype, dev)
    ap = _expect(lora_a, "lora_a", (L, R, K), x.dtype, dev)
    bp = _expect(lora_b, "lora_b", (L, N, R), x.dtype, dev)
    rp = _expect(row_adapter, "row_adapter", (M,), torch.int32, dev)
    sp = None if scales is None else _expect(scales, "scales", (L,), torch.float32, dev)
    kp = None if ranks is None else _expect(ranks, "ranks", (L,), torch.int32, dev)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or x.dtype, device=x.device)
    elif out.shape != (M, N) or out.get_device() != dev:
        raise ValueError(f"out must be {(M, N)} on the first tensor's device")
    if out.dtype is not x.dtype and out.dtype is not torch.float32:
        raise TypeError(f"out must be {x.dtype} or float32, not {out.dtype}")
    xs, os = x.stride(), out.stride()
    if (K > 1 and xs[1] != 1) or (N > 1 and os[1] != 1):
        raise ValueError("x and out need contiguous rows")
    ldx, ldo = (xs[0], os[0]) if M else (max(K, 1), max(N, 1))
    ws, nbytes, keep = _workspace(workspace, dev, lora_workspace, M, K, R)
    _run(dev, lib().tcm_lora_gemm_tn, x.data_ptr(), ldx, wp, ap, bp, rp, kp, sp, out.data_ptr(), ldo,
         M, N, K, L, R, code, _OUT[out.dtype], ws, nbytes)
    return out


def qk_norm_rope(q, k, positions, inv_freq, wq=None, wk=None, eps=1e-6, layout="half", factor=1.0,
                 norm=True, q_out=None, k_out=None):
    """(q_out, k_out): the heads of q (T, Hq, D) and k (T, Hk, D), float16/bfloat16
    views with contiguous heads, normed (n = x w / sqrt(mean(x^2) + eps); norm=False:
    n = x) and their first 2 len(inv_freq) elements rotated by positions[t] *
    inv_freq[j] and scaled by factor.  positions (T,) int32, inv_freq float64
    (rope_frequencies) or None; layout "half" (pairs j, j + rot/2) or
    "interleaved" (2j, 2j + 1); wq, wk (D,) of q's type or float32.  q_out may be q
    and k_out k."""
    code = _half(q, "q")
    dev, dt = q.get_device(), q.dtype
    T, Hq, D = q.shape
    Hk = k.shape[1]
    qs, ks = (T, Hq, D), (T, Hk, D)
    if q_out is None:
        q_out = torch.empty(qs, dtype=dt, device=q.device)
    if k_out is None:
        k_out = torch.empty(ks, dtype=dt, device=q.device)
    r = _rope(T, D, positions, inv_freq, wq, wk, eps, layout, factor, norm, dt, dev)
    _run(dev, lib().tcm_qk_norm_rope, _heads(q, "q", qs, dt, dev),
         _heads(k, "k", ks, dt, dev), _heads(q_out, "q_out", qs, dt, dev),
         _heads(k_out, "k_out", ks, dt, dev), T, Hq, Hk, r, code)
    return q_out, k_out


def qk_norm_rope_cache(q, k, v, positions, inv_freq, k_cache, v_cache, slots, wq=None, wk=None,
                       eps=1e-6, layout="half", factor=1.0, norm=True, k_scale=1.0, v_scale=1.0,
                       q_out=None):
    """q_out as qk_norm_rope; the normed and rotated keys and the values v (T, Hk, D)
    go into the caches (pages, page_size, Hk, D) at slots[t] = page * page_size +
    place (int32; outside the cache, -1 by custom: nothing is written).  Caches are
    of q's type, or E4M3 (float8_e4m3fn or uint8), which holds k / k_scale and
    v / v_scale."""
    code = _half(q, "q")
    dev, dt = q.get_device(), q.dtype
    T, Hq, D = q.shape
    Hk = k.shape[1]
    qs, ks = (T, Hq, D), (T, Hk, D)
    if q_out is None:
        q_out = torch.empty(qs, dtype=dt, device=q.device)
    r = _rope(T, D, positions, inv_freq, wq, wk, eps, layout, factor, norm, dt, dev)
    _run(dev, lib().tcm_qk_norm_rope_cache, _heads(q, "q", qs, dt, dev),
         _heads(k, "k", ks, dt, dev), _heads(v, "v", ks, dt, dev),
         _heads(q_out, "q_out", qs, dt, dev),
         _cache(k_cache, v_cache, k_scale, v_scale, Hk, D, dt, dev),
         _expect(slots, "slots", (T,), torch.int32, dev), T, Hq, Hk, r, code)
    return q_out


def qk_norm_rope_bwd_workspace(D):
    """Bytes of workspace of qk_norm_rope_bwd."""
    return _bytes(lib().tcm_qk_norm_rope_bwd_workspace, D)


def qk_norm_rope_bwd(dq_out, dk_out, q, k, positions, inv_freq, wq=None, wk=None, eps=1e-6,
                     layout="half", factor=1.0, norm=True, dq=None, dk=None, dwq=None, dwk=None,
                     workspace=None):
    """(dq, dk, dwq, dwk): the gradients of qk_norm_rope's inputs and weights from
    those of its outputs; q, k and the rest as given to it.  dwq, dwk (D,) float32
    are computed for the weights that are given (else None)."""
    code = _half(q, "q")
    dev, dt = q.get_device(), q.dtype
    T, Hq, D = q.shape
    Hk = k.shape[1]
    qs, ks = (T, Hq, D), (T, Hk, D)
    if dq is None:
        dq = torch.empty(qs, dtype=dt, device=q.device)
    if dk is None:
        dk = torch.empty(ks, dtype=dt, device=q.device)
    r = _rope(T, D, positions, inv_freq, wq, wk, eps, layout, factor, norm, dt, dev)
    if wq is None:
        dwq = None
    elif dwq is None:
        dwq = torch.empty((D,), dtype=torch.float32, device=q.device)
    if wk is None:
        dwk = None
    elif dwk is None:
        dwk = torch.empty((D,), dtype=torch.float32, device=q.device)
    ws = nbytes = keep = None
    if dwq is not None or dwk is not None:
        ws, nbytes, keep = _workspace(workspace, dev, qk_norm_rope_bwd_workspace, D)
    _run(dev, lib().tcm_qk_norm_rope_bwd, _heads(dq_out, "dq_out", qs, dt, dev),
         _heads(dk_out, "dk_out", ks, dt, dev), _heads(q, "q", qs, dt, dev),
         _heads(k, "k", ks, dt, dev), _heads(dq, "dq", qs, dt, dev),
         _heads(dk, "dk", ks, dt, dev),
         None if dwq is None else _expect(dwq, "dwq", (D,), torch.float32, dev),
         None if dwk is None else _expect(dwk, "dwk", (D,), torch.float32, dev), T, Hq, Hk, r, code, ws,
         nbytes or 0)
    return dq, dk, dwq, dwk


def paged_attention_workspace(B, Hq, Hk, D, max_len):
    """Bytes of workspace of paged_attention, for at most B sequences of lengths up to
    max_len and every window."""
    return _bytes(lib().tcm_paged_attention_workspace, B, Hq, Hk, D, max_len)


def paged_attention(q, k_cache, v_cache, block_table, lengths, scale=None, window=0, max_len=None,
                    k_scale=1.0, v_scale=1.0, out=None, lse=None, workspace=None):
    """out (B, Hq, D): softmax(scale q k^T) v of one new token per sequence, q
    (B, Hq, D) float16/bfloat16, over the keys of sequence b in the caches (pages,
    page_size, Hk, D): key j at place j % page_size of page block_table[b, j //
    page_size] (int32; an entry outside the cache is a hole, whose keys are not
    attended).  lengths (B,) int32; window > 0: the last `window` keys only;
    scale: 1 / sqrt(D) if None; max_len: an upper bound of the lengths (the
    table's room if None), which the split over the length goes by.  A sequence
    without keys gives zeros.  lse (B, Hq) float32 takes the logarithm of the sum
    of exponentials (-inf without keys).  out may be q."""
    code = _half(q, "q")
    dev, dt = q.get_device(), q.dtype
    qs = B, Hq, D = tuple(q.shape)
    _, page_size, Hk, _ = k_cache.shape
    if out is None:
        out = torch.empty(qs, dtype=dt, device=q.device)
    if block_table.dim() != 2 or block_table.shape[0] != B or block_table.dtype is not torch.int32:
        raise ValueError(f"block_table must be ({B}, pages of a sequence) int32")
    per, (ts, es) = block_table.shape[1], block_table.stride()
    if block_table.get_device() != dev or (per > 1 and es != 1) or (B > 1 and ts < per):
        raise ValueError("block_table must have contiguous rows and be on the first tensor's device")
    if max_len is None or max_len > per * page_size:
        max_len = per * page_size
    cache = _cache(k_cache, v_cache, k_scale, v_scale, Hk, D, dt, dev)
    ws, nbytes, keep = _workspace(workspace, dev, paged_attention_workspace, B, Hq, Hk, D, max_len)
    _run(dev, lib().tcm_paged_attention, _heads(q, "q", qs, dt, dev), cache, block_table.data_ptr(),
         ts if B > 1 and per else per, _expect(lengths, "lengths", (B,), torch.int32, dev), max_len,
         _heads(out, "out", qs, dt, dev),
         None if lse is None else _expect(lse, "lse", (B, Hq), torch.float32, dev), B, Hq, Hk, D,
         D ** -0.5 if scale is None else scale, window, code, ws, nbytes)
    return out


def rope_frequencies(rot_dim, base=10000.0, scaling=None, ratio=1.0, trained=None, low=1.0, high=32.0,
                     device="cpu"):
    """(inv_freq, factor) of the rotation of rot_dim elements: inv_freq[j] =
    base^(-2j / rot_dim), a float64 tensor of rot_dim / 2, and the factor 1; or, to
    stretch a context of `trained` positions `ratio` times,

    * "linear": every frequency divided by ratio (positions interpolated);
    * "ntk":    base * ratio^(rot_dim / (rot_dim - 2)): the lowest frequency is
                divided by ratio and the highest kept;
    * "yarn":   frequency j keeps the share g_j and is divided by ratio for the rest;
                with c_j = trained * inv_freq[j] / 2 pi turns over the trained
                context, the index of c turns is i(c) = rot_dim / 2 * log(trained /
                (2 pi c)) / log(base), and g falls linearly over the indices from 1 at
                floor(i(high)) to 0 at ceil(i(low)); factor = 0.1 log(ratio) + 1;
    * "bands":  g_j rises linearly in c_j itself, from 0 at `low` turns to 1 at
                `high`; factor 1.
    """
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even")
    j = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "ntk":
        if rot_dim <= 2:
            raise ValueError("ntk scaling needs more than one pair")
        base = base * ratio ** (rot_dim / (rot_dim - 2))
    freq = base ** (-2.0 * j / rot_dim) if rot_dim else j
    if scaling is None or scaling == "ntk":
        return freq.to(device), 1.0
    if scaling == "linear":
        return (freq / ratio).to(device), 1.0
    if scaling not in ("yarn", "bands"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not trained or low >= high:
        raise ValueError(f"{scaling} scaling needs trained > 0 and low < high")
    if scaling == "bands":
        keep = ((trained * freq / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        return (freq * keep + freq / ratio * (1 - keep)).to(device), 1.0
    at = lambda c: rot_dim / 2 * math.log(trained / (2 * math.pi * c)) / math.log(base)  # noqa: E731
    first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot_dim - 1)
    keep = 1 - ((j - first) / max(last - first, 1e-3)).clamp(0.0, 1.0)
    return (freq * keep + freq / ratio * (1 - keep)).to(device), 0.1 * math.log(ratio) + 1.0 if ratio > 1 else 1.0
