"""paged_attention on the GPU against the float64 oracle.

Tolerance: a score is an fp32 sum of D products, off by at most (D + 4) 2^-24 of x, the
largest sum of magnitudes of its row, and so is the exponent of every probability; a
probability is rounded once to the type's precision (2^-9 bf16, 2^-12 fp16, of itself;
fp16 ones below 2^-14 of the largest by at most 2^-25 of it); sums are fp32; the output
is rounded once.
"""
import math

import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = {torch.bfloat16: "bf16", torch.float16: "f16"}
STEP = {torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12}


def f64(t):
    return t.double().cpu().numpy()


def make(B, Hq, Hk, D, lengths, page, dt, kind="same", seed=0, heads_first=False, extra=2):
    """q, caches, table (pages of a sequence anywhere, entries past its length -1)."""
    g = torch.Generator().manual_seed(seed)
    per = max(1, max(-(-n // page) for n in lengths))
    pages = B * per + extra
    shape = (pages, Hk, page, D) if heads_first else (pages, page, Hk, D)
    q = torch.randn((B, Hq, D), generator=g).to(dt).to(DEV)
    caches = []
    for _ in range(2):
        c = torch.randn(shape, generator=g)
        c = (c * 16).clamp(-448, 448).to(torch.float8_e4m3fn) if kind == "e4m3" else c.to(dt)
        c = c.to(DEV)
        caches.append(c.transpose(1, 2) if heads_first else c)
    table = torch.randperm(pages, generator=g)[: B * per].view(B, per).to(torch.int32)
    for b, n in enumerate(lengths):
        table[b, -(-n // page):] = -1
    return q, caches[0], caches[1], table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV)


def check(q, kc, vc, table, lengths, out, lse, scale=None, window=0, ks=1.0, vs=1.0):
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    page = kc.shape[1]
    k, v = f64(kc.float()) * ks, f64(vc.float()) * vs
    ref, rlse, mag, top = ol.paged_attention(f64(q), k, v, table.cpu().numpy(), lengths.tolist(), page, scale, window)
    n = int(max(lengths.tolist() + [1]))
    ds = (2 * D + 8) * 2.0 ** -24 * top + 2.0 ** -20
    rel = STEP[q.dtype] + 2 * ds[..., None] + (n // 32 + 300) * 2.0 ** -24
    tol = rel * (mag + np.abs(ref)) + 1.01 * ol.half_ulp(ref, NAMES[q.dtype])
    if q.dtype == torch.float16:
        tol += n * 2.0 ** -25 * np.abs(v).max()
    err = np.abs(f64(out) - ref)
    assert (err <= tol).all(), f"worst {np.nanmax(err / tol)} at {np.argwhere(~(err <= tol))[:4]}"
    if lse is not None:
        got = f64(lse)
        empty = np.isneginf(rlse)
        assert (np.isneginf(got) == empty).all()
        assert (np.abs(got[~empty] - rlse[~empty]) <= (ds + 1e-5)[~empty]).all()


def run(case, **kw):
    q, kc, vc, table, lengths = case
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float32, device=DEV)
    out = torch.full(q.shape, math.nan, dtype=q.dtype, device=DEV)
    tcm.paged_attention(q, kc, vc, table, lengths, out=out, lse=lse, **kw)
    return out, lse


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 64), (4, 4, 128), (8, 1, 16), (32, 8, 128), (12, 2, 80), (6, 2, 96),
                                     (20, 1, 128), (40, 2, 64), (4, 1, 256), (33, 3, 192), (2, 2, 32)])
def test_heads(Hq, Hk, D, kind, dt):
    case = make(4, Hq, Hk, D, [1, 37, 300, 64], 16, dt, kind, Hq + D)
    kw = dict(k_scale=0.0625, v_scale=0.125) if kind == "e4m3" else {}
    out, lse = run(case, **kw)
    check(*case, out, lse, ks=kw.get("k_scale", 1.0), vs=kw.get("v_scale", 1.0))


@pytest.mark.parametrize("D", [8, 24, 72, 136, 248])
def test_head_sizes_that_fill_no_instance(D):
    case = make(2, 4, 2, D, [50, 129], 32, torch.bfloat16, seed=D)
    check(*case, *run(case))


@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("page", [1, 2, 3, 7, 8, 16, 24, 32, 48, 64, 100, 128, 512])
def test_page_sizes(page, kind):
    """Pages that end inside a tile, hold several, or are one key."""
    lengths = [1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 260, 0]
    case = make(len(lengths), 4, 2, 64, lengths, page, torch.float16, kind, page)
    check(*case, *run(case))


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("B,n", [(1, 1), (1, 257), (1, 5000), (1, 40001), (2, 3000), (3, 9000), (40, 700)])
def test_split_over_the_length(B, n, heads_first):
    """Ragged lengths, most of them far below the longest: chunks without a key, joins of
    one and of many."""
    lengths = [max(0, n - 397 * b * b) for b in range(B)]
    case = make(B, 8, 2, 64, lengths, 64, torch.bfloat16, seed=n, heads_first=heads_first)
    check(*case, *run(case))
    if n == 5000:  # an upper bound that is no length
        check(*case, *run((*case[:3], torch.nn.functional.pad(case[3], (0, 900), value=-1), case[4])))


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("window", [1, 2, 16, 31, 33, 100, 300, 2000])
def test_windows(window, page):
    case = make(5, 4, 1, 64, [0, 1, 50, 301, 1500], page, torch.bfloat16, seed=window)
    check(*case, *run(case, window=window), window=window)


@pytest.mark.parametrize("page", [16, 64, 6])
def test_what_no_key_holds_is_not_used(page):
    """Places past a sequence's end, before its window and pages of nobody hold NaN and
    infinities; holes are passed over; a sequence of holes alone is empty."""
    lengths = [20, 333, 90, 45]
    q, kc, vc, table, n = case = make(4, 4, 2, 64, lengths, page, torch.bfloat16, seed=3)
    table[1, 2] = -1
    table[1, 4] = kc.shape[0]
    table[1, 5] = 2**31 - 1
    table[3, :] = -5
    window = 200
    live = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for b, m in enumerate(lengths):
        for j in range(max(0, m - window), m):
            p = int(table[b, j // page])
            if 0 <= p < kc.shape[0]:
                live[p, j % page] = True
    bad = ~live.to(DEV)
    clean = (q, kc.clone(), vc.clone(), table, n)
    kc[bad] = math.nan
    vc[bad] = math.inf
    out, lse = run(case, window=window)
    check(*clean, out, lse, window=window)
    assert (out[3] == 0).all() and torch.isneginf(lse[3]).all()
    kc[bad] = -math.inf
    vc[bad] = math.nan
    again, _ = run(case, window=window)
    assert torch.equal(out, again)


def test_nothing_to_attend():
    """No lengths, negative ones, no pages at all, a table without columns."""
    q, kc, vc, table, n = make(3, 4, 2, 64, [5, 5, 5], 16, torch.bfloat16)
    zero = torch.tensor([0, -3, -2**31], dtype=torch.int32, device=DEV)
    for case in ((q, kc, vc, table, zero), (q, kc[:0], vc[:0], table, n), (q, kc, vc, table[:, :0], n)):
        out, lse = run(case)
        assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = run((q, kc, vc, table, n), max_len=0)
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert tcm.paged_attention(q[:0], kc, vc, table[:0], n[:0]).shape == (0, 4, 64)


def test_lengths_beyond_the_table_are_clipped():
    case = make(2, 4, 2, 64, [30, 64], 16, torch.bfloat16, seed=4)
    long = torch.tensor([30, 2**31 - 1], dtype=torch.int32, device=DEV)
    out, lse = run((*case[:4], long))
    check(*case, out, lse)
    short = torch.tensor([30, 40], dtype=torch.int32, device=DEV)
    out, lse = run((*case[:4], long), max_len=40)
    check(*case[:4], short, out, lse)


def test_queries_that_are_not_finite_and_large_scores():
    q, kc, vc, table, n = case = make(3, 4, 2, 64, [40, 600, 3], 16, torch.bfloat16, seed=5)
    want, wl = run(case)
    q2 = q.clone()
    q2[1, 2, 7] = math.nan
    q2[2, 1, 0] = math.inf
    got, gl = run((q2, kc, vc, table, n))
    assert torch.isnan(got[1, 2]).all() and torch.isnan(gl[1, 2]) and torch.isnan(got[2, 1]).all()
    for b, h in ((1, 2), (2, 1)):
        got[b, h], gl[b, h] = want[b, h], wl[b, h]
    assert torch.equal(got, want) and torch.equal(gl, wl)
    # scores of +-1e4: one key takes all, nothing overflows
    out, lse = run(case, scale=1000.0)
    check(*case, out, lse, scale=1000.0)
    out, lse = run(case, scale=-0.7)
    check(*case, out, lse, scale=-0.7)


def test_every_e4m3_code_is_the_value_it_stands_for():
    """One key a sequence: the output is its value."""
    codes = torch.arange(256, dtype=torch.uint8, device=DEV)
    vc = codes.view(16, 1, 1, 16).contiguous()
    kc = torch.zeros_like(vc)
    for dt in NAMES:
        q = torch.ones((16, 1, 16), dtype=dt, device=DEV)
        table = torch.arange(16, dtype=torch.int32, device=DEV).view(16, 1)
        n = torch.ones(16, dtype=torch.int32, device=DEV)
        out = tcm.paged_attention(q, kc, vc, table, n, v_scale=0.5).view(-1).float()
        want = codes.view(torch.float8_e4m3fn).float() * 0.5
        assert torch.equal(torch.nan_to_num(out, nan=1e9), torch.nan_to_num(want, nan=1e9))


def test_strides_alias_and_workspace():
    """q a slice of a fused projection, out = q, a table that is a slice of a wider one, a
    dirty workspace: the same bits."""
    B, Hq, Hk, D = 3, 8, 2, 128
    q, kc, vc, table, n = make(B, Hq, Hk, D, [2000, 77, 900], 16, torch.bfloat16, seed=6)
    want, _ = run((q, kc, vc, table, n))
    wide = torch.zeros((B, Hq + 4, D), dtype=torch.bfloat16, device=DEV)
    wide[:, 2:2 + Hq] = q
    view = wide[:, 2:2 + Hq]
    t2 = torch.full((B, table.shape[1] + 9), 0, dtype=torch.int32, device=DEV)
    t2[:, 4:4 + table.shape[1]] = table
    need = tcm.paged_attention_workspace(B, Hq, Hk, D, 2000)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    got = tcm.paged_attention(view, kc, vc, t2[:, 4:4 + table.shape[1]], n, max_len=2000, out=view, workspace=ws)
    assert got.data_ptr() == view.data_ptr()
    ref = tcm.paged_attention(q, kc, vc, table, n, max_len=2000)
    assert torch.equal(got, ref)
    check(q, kc, vc, table, n, want, None)
    assert (wide[:, :2] == 0).all() and (wide[:, 2 + Hq:] == 0).all()
    with pytest.raises(tcm.TcmError):
        tcm.paged_attention(q, kc, vc, table, n, max_len=2000, workspace=ws[: need // 8 // 16 * 16])


def test_cache_of_more_than_2_to_31_elements():
    """Pages whose offsets pass 32 bits (4.3 GiB of keys)."""
    Hk, D, page = 8, 128, 64
    pages = (1 << 31) // (page * Hk * D) + 40
    kc = torch.zeros((pages, page, Hk, D), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    g = torch.Generator(device=DEV).manual_seed(1)
    far = [pages - 1, pages - 17, 3]
    for p in far:
        kc[p] = torch.randn((page, Hk, D), generator=g, device=DEV).to(torch.bfloat16)
        vc[p] = torch.randn((page, Hk, D), generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn((1, 16, D), generator=g, device=DEV).to(torch.bfloat16)
    table = torch.tensor([far], dtype=torch.int32, device=DEV)
    n = torch.tensor([150], dtype=torch.int32, device=DEV)
    out, lse = run((q, kc, vc, table, n))
    small = (q, kc[far].contiguous(), vc[far].contiguous(),
             torch.arange(3, dtype=torch.int32, device=DEV).view(1, 3), n)
    check(*small, out, lse)
