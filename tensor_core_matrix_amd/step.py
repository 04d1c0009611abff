"""A step that drafts several tokens at once: pages and slots for them, the residual sum and
norm before a product, products of few rows with 4-bit weights, and the attention of the
drafted tokens over the paged cache (C ABI in ``include/tcm.h``).

Tensors, streams and workspaces as in ``layer.py``.
"""
from __future__ import annotations

import torch

from . import E2M1, F32, U4, lib
from .layer import _OUT, _bytes, _cache, _expect, _half, _heads, _run, _workspace

__all__ = ["cache_plan", "add_rms_norm", "add_rms_norm_mx_fp8", "add_rms_norm_bwd",
           "add_rms_norm_bwd_workspace", "gemm_w4", "paged_tree_attention",
           "paged_tree_attention_workspace"]

_MX = {"elements": (torch.float8_e4m3fn, torch.uint8), "scales": (torch.float8_e8m0fnu, torch.uint8)}


def _table(t, B, dev):
    """(address, row stride, width) of a block table of B rows."""
    if t.dim() != 2 or t.shape[0] != B or t.dtype is not torch.int32:
        raise ValueError(f"block_table must be ({B}, pages of a sequence) int32")
    per, (ts, es) = t.shape[1], t.stride()
    if t.get_device() != dev or (per > 1 and es != 1) or (B > 1 and ts < per):
        raise ValueError("block_table must have contiguous rows and be on the first tensor's device")
    return t.data_ptr(), ts if B > 1 and per else per, per


def cache_plan(lengths, change, block_table, free_pages, free_count, page_size, tokens=None, pages=None,
               starts=None, slots=None, positions=None, missing=None):
    """(starts, slots, positions) of the new tokens when the B sequences of a paged cache change their
    lengths by change[b]: more keys (drafts, a prompt) or fewer (drafts that were refused; all: the
    request has ended).  lengths (B,), block_table (B, pages of a sequence), the stack free_pages
    (pages,) of which the first free_count (1,) entries are free pages, its last one the top, are
    updated: entries of pages that hold no key any more become -1 and their pages go back on the
    stack; new ones come from its top, -1 when there is none (missing (1,), if given, takes how many).
    The opposite changes right after put everything back.  starts (B + 1,): token starts[b] + i is
    sequence b's new token i; slots and positions (tokens,) as qk_norm_rope_cache takes them, slot -1
    for a token without a page and behind the last token.  All int32; `tokens` is the room for new
    tokens (those of slots, if given), pages the cache's pages (len(free_pages) if None)."""
    dev = lengths.get_device()
    B = lengths.shape[0]
    i32 = torch.int32
    lp = _expect(lengths, "lengths", (B,), i32, dev)
    cp = _expect(change, "change", (B,), i32, dev)
    tp, ts, per = _table(block_table, B, dev)
    capacity = free_pages.numel()
    fp = _expect(free_pages, "free_pages", (capacity,), i32, dev)
    np = _expect(free_count, "free_count", (1,), i32, dev)
    if tokens is None:
        if slots is None and positions is None:
            raise ValueError("tokens: the room for new tokens")
        tokens = (slots if slots is not None else positions).shape[0]
    new = lambda n: torch.empty((n,), dtype=i32, device=lengths.device)  # noqa: E731
    starts = new(B + 1) if starts is None else starts
    slots = new(tokens) if slots is None else slots
    positions = new(tokens) if positions is None else positions
    _run(dev, lib().tcm_cache_plan, lp, cp, tp, ts, per, B, capacity if pages is None else pages, page_size, fp,
         capacity, np, _expect(starts, "starts", (B + 1,), i32, dev), _expect(slots, "slots", (tokens,), i32, dev),
         _expect(positions, "positions", (tokens,), i32, dev), tokens,
         None if missing is None else _expect(missing, "missing", (1,), i32, dev))
    return starts, slots, positions


def _rows(t, what, shape, dtypes, dev):
    """(address, row stride) of a (T, D) tensor with contiguous rows."""
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(map(str, dtypes))}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    s = t.stride()
    if t.get_device() != dev or (shape[1] > 1 and s[1] != 1):
        raise ValueError(f"{what} must have contiguous rows and be on the first tensor's device")
    return t.data_ptr(), s[0]


def _weight(w, D, dtype, dev):
    """(address, type code) of a norm's weight."""
    if w is None:
        return None, F32
    if w.dtype is not dtype and w.dtype is not torch.float32:
        raise TypeError(f"weight must be {dtype} or float32, not {w.dtype}")
    return _expect(w, "weight", (D,), w.dtype, dev), _OUT[w.dtype]


def _summed(x, residual, sum_out, shape, dev, out=None):
    """(x, residual, sum) as (address, stride) pairs, and the sum's tensor: x itself where nothing is added to it
    and out does not overwrite it."""
    dt = (x.dtype,)
    onto = out is not None and x.numel() > 0 and out.data_ptr() == x.data_ptr()
    if sum_out is None and (residual is not None or onto):
        sum_out = torch.empty(shape, dtype=x.dtype, device=x.device)
    none = (None, 0)
    return (_rows(x, "x", shape, dt, dev), none if residual is None else _rows(residual, "residual", shape, dt, dev),
            none if sum_out is None else _rows(sum_out, "sum_out", shape, dt, dev),
            x if sum_out is None else sum_out)


def add_rms_norm(x, weight=None, residual=None, eps=1e-6, out=None, out_dtype=None, sum_out=None):
    """(out, s): s = x + residual (x without one) rounded to x's type, and out = weight s / sqrt(mean(s^2) +
    eps) for every row, of s before it is rounded.  x, residual, s (T, D) float16/bfloat16 with contiguous rows; weight
    (D,) of x's type or float32; out of x's type or float32.  sum_out and out may be x or residual; without a residual
    and sum_out s is x itself, or a copy of it where out is x."""
    code = _half(x, "x")
    dev = x.get_device()
    T, D = shape = x.shape
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or x.dtype, device=x.device)
    (xp, ldx), (rp, ldr), (sp, lds), s = _summed(x, residual, sum_out, shape, dev, out)
    op, ldo = _rows(out, "out", shape, (x.dtype, torch.float32), dev)
    wp, wt = _weight(weight, D, x.dtype, dev)
    _run(dev, lib().tcm_add_rms_norm, xp, ldx, rp, ldr, wp, wt, eps, sp, lds, op, ldo, T, D, code, _OUT[out.dtype])
    return out, s


def add_rms_norm_mx_fp8(x, weight=None, residual=None, eps=1e-6, out=None, scale=None, sum_out=None):
    """(out, scale, s): add_rms_norm with the result in MXFP8, as gemm_mx_fp8 takes it: out (T, D)
    E4M3 (float8_e4m3fn, or uint8) and scale (T, D / 32) E8M0 (uint8, or float8_e8m0fnu), the
    smallest power of two that takes the 32 elements to at most 448."""
    code = _half(x, "x")
    dev = x.get_device()
    T, D = shape = x.shape
    if out is None:
        out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
    if scale is None:
        scale = torch.empty((T, D // 32), dtype=torch.uint8, device=x.device)
    for t, what, n in ((out, "elements", D), (scale, "scales", D // 32)):
        if t.dtype not in _MX[what]:
            raise TypeError(f"{what} must be {' or '.join(map(str, _MX[what]))}, not {t.dtype}")
        _expect(t, what, (T, n), t.dtype, dev)
    (xp, ldx), (rp, ldr), (sp, lds), s = _summed(x, residual, sum_out, shape, dev)
    wp, wt = _weight(weight, D, x.dtype, dev)
    _run(dev, lib().tcm_add_rms_norm_mx_fp8, xp, ldx, rp, ldr, wp, wt, eps, sp, lds, out.data_ptr(),
         scale.data_ptr(), T, D, code)
    return out, scale, s


def add_rms_norm_bwd_workspace(T, D):
    """Bytes of workspace of add_rms_norm_bwd, enough also for fewer rows."""
    return _bytes(lib().tcm_add_rms_norm_bwd_workspace, T, D)


def add_rms_norm_bwd(dout, s, weight=None, dsum=None, eps=1e-6, dx=None, dw=None, workspace=None):
    """(dx, dw): the gradients of add_rms_norm's x (and of its residual: the same) and of its weight, from
    those of its results, dout and dsum (None: none), and the sum s that it kept.  dw (D,)
    float32 is computed if there is a weight (else None)."""
    code = _half(dout, "dout")
    dev, dt = dout.get_device(), (dout.dtype,)
    T, D = shape = dout.shape
    if dx is None:
        dx = torch.empty(shape, dtype=dout.dtype, device=dout.device)
    if weight is None:
        dw = None
    elif dw is None:
        dw = torch.empty((D,), dtype=torch.float32, device=dout.device)
    dp, ldd = _rows(dout, "dout", shape, dt, dev)
    sp, lds = _rows(s, "s", shape, dt, dev)
    gp, ldg = (None, 0) if dsum is None else _rows(dsum, "dsum", shape, dt, dev)
    xp, ldx = _rows(dx, "dx", shape, dt, dev)
    wp, wt = _weight(weight, D, dout.dtype, dev)
    ws = nbytes = keep = None
    if dw is not None:
        ws, nbytes, keep = _workspace(workspace, dev, add_rms_norm_bwd_workspace, T, D)
    _run(dev, lib().tcm_add_rms_norm_bwd, dp, ldd, gp, ldg, sp, lds, wp, wt, eps, xp, ldx,
         None if dw is None else _expect(dw, "dw", (D,), torch.float32, dev), T, D, code, ws, nbytes or 0)
    return dx, dw


_ELEMS = {"u4": U4, "e2m1": E2M1}


def gemm_w4(x, w, scales, zeros=None, elem="u4", out=None, out_dtype=None):
    """out = x . W^T for few rows x (M, K), float16/bfloat16 with contiguous rows, and 4-bit
    weights w (N, K/2) uint8, element 2t in the low four bits of byte t.
    elem "u4": W = scales[n, g] (q - zeros[n, g]), q = 0 .. 15, groups g of K / scales.shape[1] values (a
    multiple of 32), scales (N, groups) of x's type, zeros (N, groups) uint8 or None (8).
    elem "e2m1": E2M1 elements times 2^(scales - 127), scales (N, K / 32) E8M0 (uint8 or
    float8_e8m0fnu): the weights of gemm_mx_fp4.
    out (M, N) of x's type or float32, with contiguous rows."""
    code = _half(x, "x")
    dev = x.get_device()
    M, K = x.shape
    N = w.shape[0]
    kind = _ELEMS.get(elem)
    if kind is None:
        raise ValueError(f"elem must be one of {sorted(_ELEMS)}, not {elem!r}")
    wp = _expect(w, "w", (N, K // 2), torch.uint8, dev)
    groups = scales.shape[1] if scales.dim() == 2 else 0
    if K and (groups < 1 or K % groups):
        raise ValueError(f"scales must be ({N}, groups) with groups of K / groups values")
    if elem == "e2m1":
        if scales.dtype not in _MX["scales"]:
            raise TypeError(f"scales must be {' or '.join(map(str, _MX['scales']))}, not {scales.dtype}")
        sp = _expect(scales, "scales", (N, K // 32), scales.dtype, dev)
    else:
        sp = _expect(scales, "scales", (N, groups), x.dtype, dev)
    zp = None if zeros is None else _expect(zeros, "zeros", (N, groups), torch.uint8, dev)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or x.dtype, device=x.device)
    xp, ldx = _rows(x, "x", (M, K), (x.dtype,), dev)
    op, ldo = _rows(out, "out", (M, N), (x.dtype, torch.float32), dev)
    _run(dev, lib().tcm_gemm_w4, xp, ldx, wp, sp, zp, op, ldo, M, N, K, K // groups if K else 32, kind, code,
         _OUT[out.dtype])
    return out


def paged_tree_attention_workspace(B, Hq, Hk, D, max_nodes, max_len):
    """Bytes of workspace of paged_tree_attention, for at most B sequences of at most max_nodes new tokens
    and lengths up to max_len, and every window."""
    return _bytes(lib().tcm_paged_tree_attention_workspace, B, Hq, Hk, D, max_nodes, max_len)


def paged_tree_attention(q, k_cache, v_cache, block_table, lengths, starts, max_nodes, tree=None, scale=None,
                         window=0, max_len=None, k_scale=1.0, v_scale=1.0, out=None, lse=None, workspace=None):
    """out (T, Hq, D): attention of several new tokens per sequence, q (T, Hq, D), over the paged cache
    that holds their keys and values already.  Rows starts[b] .. starts[b + 1] - 1 (starts (B + 1,)
    int32, as cache_plan gives it; at most max_nodes a sequence) are the last keys of sequence b, of
    lengths[b] keys in all.  tree None: a chain, each token sees what is before it and itself.  tree
    (T, words) int64: each sees the keys before the sequence's new tokens, and of those the
    ones whose bits are set (token j: bit j % 64 of word j // 64; itself among them).  window > 0: of a
    chain the last `window` keys of each token; of a tree's context the keys less than `window` places
    before the token, which is as many places behind the context as it has bits.  Rows of no sequence are left
    as they were; a row that sees nothing gives zeros.  The rest as paged_attention, lse (T, Hq)."""
    code = _half(q, "q")
    dev, dt = q.get_device(), q.dtype
    qs = T, Hq, D = tuple(q.shape)
    _, page_size, Hk, _ = k_cache.shape
    B = lengths.shape[0]
    if out is None:
        out = torch.empty(qs, dtype=dt, device=q.device)
    tp, ts, per = _table(block_table, B, dev)
    if max_len is None or max_len > per * page_size:
        max_len = per * page_size
    words = 0
    if tree is not None:
        if tree.dim() != 2:
            raise ValueError(f"tree must be ({T}, words) int64")
        words = tree.shape[1]
        if 64 * words < max_nodes:  # (none at all would have no address, and be a chain)
            raise ValueError(f"tree must have a bit for each of {max_nodes} tokens, not {words} words")
        tree = _expect(tree, "tree", (T, words), torch.int64, dev)
    cache = _cache(k_cache, v_cache, k_scale, v_scale, Hk, D, dt, dev)
    ws, nbytes, keep = _workspace(workspace, dev, paged_tree_attention_workspace, B, Hq, Hk, D, max_nodes, max_len)
    _run(dev, lib().tcm_paged_tree_attention, _heads(q, "q", qs, dt, dev), cache, tp, ts,
         _expect(lengths, "lengths", (B,), torch.int32, dev), max_len,
         _expect(starts, "starts", (B + 1,), torch.int32, dev), max_nodes, tree, words,
         _heads(out, "out", qs, dt, dev), None if lse is None else _expect(lse, "lse", (T, Hq), torch.float32, dev),
         T, B, Hq, Hk, D, D ** -0.5 if scale is None else scale, window, code, ws, nbytes)
    return out
