"""paged_tree_attention on the GPU against the float64 oracle.

Tolerance: a score is an fp32 sum of D products, off by at most (D + 4) 2^-24 of x, the largest
sum of magnitudes of its row, and so is the exponent of every probability; a probability enters as two
16-bit parts, 2^-16 of itself together (bf16) or 2^-22; sums are fp32; the output is rounded once.
"""
import math
import random

import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol
from oracle import step as os_

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
NAMES = {BF: "bf16", HF: "f16"}


def f64(t):
    return t.double().cpu().numpy()


def random_tree(m, r):
    """Bits of m nodes that hang on an earlier one or on the context."""
    rows = []
    for i in range(m):
        up = r.randrange(-1, i) if i else -1
        rows.append((rows[up] if up >= 0 else 0) | 1 << i)
    return rows


def make(Hq, Hk, D, lengths, nodes, page, dt, kind="same", seed=0, tree=True, behind=3, words=None, heads_first=False):
    """A case: the call's tensors, and the tree's rows as Python ints."""
    g, r = torch.Generator().manual_seed(seed), random.Random(seed)
    B = len(lengths)
    per = max(1, max(-(-n // page) for n in lengths))
    pages = B * per + 2
    T = sum(nodes) + behind
    q = torch.randn((T, Hq, D), generator=g).to(dt).to(DEV)
    caches = []
    for _ in range(2):
        c = torch.randn((pages, Hk, page, D) if heads_first else (pages, page, Hk, D), generator=g)
        c = ((c * 16).clamp(-448, 448).to(torch.float8_e4m3fn) if kind == "e4m3" else c.to(dt)).to(DEV)
        caches.append(c.transpose(1, 2) if heads_first else c)
    table = torch.randperm(pages, generator=g)[: B * per].view(B, per).to(torch.int32)
    for b, n in enumerate(lengths):
        table[b, -(-n // page):] = -1
    starts = [sum(nodes[:b]) for b in range(B + 1)]
    bits = None
    if tree:
        bits = [x for m in nodes for x in random_tree(m, r)] + [r.getrandbits(64) for _ in range(behind)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(q=q, k=caches[0], v=caches[1], table=table.to(DEV), lengths=i32(lengths), starts=i32(starts), bits=bits,
                max_nodes=max(nodes + [1]), words=words or -(-max(nodes + [1]) // 64),
                ks=0.0625 if kind == "e4m3" else 1.0, vs=0.125 if kind == "e4m3" else 1.0)


def tree_tensor(bits, words):
    half = 1 << 63
    return torch.tensor([[((x >> 64 * w) + half) % (1 << 64) - half for w in range(words)] for x in bits], dtype=torch.int64,
                        device=DEV)


def run(c, **kw):
    lse = torch.full(c["q"].shape[:2], 9.0, dtype=torch.float32, device=DEV)
    out = torch.full(c["q"].shape, 7.0, dtype=c["q"].dtype, device=DEV)
    tree = None if c["bits"] is None else tree_tensor(c["bits"], c["words"])
    tcm.paged_tree_attention(c["q"], c["k"], c["v"], c["table"], c["lengths"], c["starts"], c["max_nodes"], tree=tree,
                             k_scale=c["ks"], v_scale=c["vs"], out=out, lse=lse, **kw)
    return out, lse


def check(c, out, lse, window=0, scale=None, max_nodes=None):
    T, Hq, D = c["q"].shape
    scale = D ** -0.5 if scale is None else scale
    ref = os_.tree_attention(f64(c["q"]), f64(c["k"].float()) * c["ks"], f64(c["v"].float()) * c["vs"], c["table"].cpu().numpy(),
                             c["lengths"].tolist(), c["starts"].tolist(), c["k"].shape[1], scale, c["bits"], window,
                             max_nodes or c["max_nodes"])
    n = max(c["lengths"].tolist())
    rest = [t for t in range(T) if t not in ref]
    assert (out[rest] == 7).all() and (lse[rest] == 9).all()
    got, glse = f64(out), f64(lse)
    for t, (o, l, mag, top) in ref.items():
        ds = (2 * D + 8) * 2.0 ** -24 * top + 2.0 ** -20
        rel = 2.0 ** -16 + 2 * ds[:, None] + (n // 32 + 300) * 2.0 ** -24
        tol = rel * (mag + np.abs(o)) + 1.01 * ol.half_ulp(o, NAMES[c["q"].dtype])
        err = np.abs(got[t] - o)
        assert (err <= tol).all(), (t, np.nanmax(err / tol))
        empty = np.isneginf(l)
        assert (np.isneginf(glse[t]) == empty).all()
        assert (np.abs(glse[t] - l)[~empty] <= (ds + 1e-5)[~empty]).all(), t


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 64), (4, 4, 128), (8, 1, 16), (32, 8, 128), (12, 2, 80), (6, 2, 96),
                                     (20, 1, 128), (4, 1, 256), (33, 3, 192), (2, 2, 32)])
def test_heads(Hq, Hk, D, kind, dt, tree):
    c = make(Hq, Hk, D, [6, 37, 300, 64], [6, 3, 7, 1], 16, dt, kind, Hq + D, tree)
    check(c, *run(c))


@pytest.mark.parametrize("D", [8, 24, 72, 136, 248])
@pytest.mark.parametrize("m", [2, 20])
def test_head_sizes_that_fill_no_instance(D, m):
    c = make(4, 2, D, [50, 129], [m, m - 1], 32, BF, seed=D)
    check(c, *run(c))


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("nodes", [[1], [4], [5, 0, 3], [16, 15], [17], [31, 33], [64, 1, 40], [65], [130, 64]])
@pytest.mark.parametrize("G", [1, 4])
def test_tokens(nodes, G, kind, tree):
    """Numbers of rows on both sides of every block's size; trees of more than one word."""
    lengths = [m + 41 * (b + 1) for b, m in enumerate(nodes)]
    c = make(2 * G, 2, 64, lengths, nodes, 16, BF, kind, sum(nodes), tree)
    check(c, *run(c))


@pytest.mark.parametrize("D,kind", [(128, "same"), (128, "e4m3"), (256, "same"), (256, "e4m3"), (64, "same")])
@pytest.mark.parametrize("m", [2, 12, 40])
def test_tokens_of_large_heads(m, D, kind):
    c = make(8, 2, D, [700, m, 90 + m], [m, m, 1], 16, HF, kind, m)
    check(c, *run(c))


@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("m", [3, 30])
@pytest.mark.parametrize("page", [1, 2, 3, 7, 8, 16, 24, 32, 48, 64, 100, 128, 512])
def test_page_sizes(page, m, kind):
    lengths = [m, m + 1, 31, 32, 33, 63, 64, 65, 260, 0]
    nodes = [min(m, n) for n in lengths]
    c = make(4, 2, 64, lengths, nodes, page, HF, kind, page)
    check(c, *run(c))


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("B,n,m", [(1, 5000, 4), (1, 40001, 2), (2, 3000, 20), (3, 9000, 9), (30, 700, 3)])
def test_split_over_the_length(B, n, m, heads_first):
    lengths = [max(m, n - 397 * b * b) for b in range(B)]
    c = make(8, 2, 64, lengths, [m] * B, 64, BF, seed=n, heads_first=heads_first)
    check(c, *run(c))
    if n == 5000:  # upper bounds that no sequence reaches
        c["table"] = torch.nn.functional.pad(c["table"], (0, 900), value=-1)
        c["max_nodes"], c["words"] = 150, 3
        check(c, *run(c))


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("window", [1, 2, 7, 16, 31, 33, 100, 300, 2000])
def test_windows(window, page, tree):
    for nodes, seed in (([0, 1, 5, 9, 3], window), ([20, 70, 1, 33, 64], window + 1)):
        lengths = [nodes[0], 70, 50, 301, 1500]
        c = make(4, 1, 64, lengths, nodes, page, BF, seed=seed, tree=tree)
        check(c, *run(c, window=window), window=window)


def test_rows_that_see_nothing():
    """Trees whose rows mark nothing, or not themselves, without a context and with one."""
    c = make(4, 2, 64, [5, 30], [5, 4], 16, BF)
    c["bits"][:5] = [0, 1, 0, 0b10, 0]
    c["bits"][5:9] = [0, 0b1000, 0xF, -1 & (1 << 64) - 1]  # (bits past a sequence's tokens mean nothing)
    out, lse = run(c)
    check(c, out, lse)
    assert (out[0] == 0).all() and torch.isneginf(lse[[0, 2, 4]]).all()
    check(c, *run(c, window=3), window=3)


def test_lengths_and_starts_that_do_not_fit():
    """More tokens than keys, than max_nodes and than rows; starts that go on past the rows."""
    c = make(4, 2, 64, [3, 40, 20, 9], [5, 9, 20, 4], 16, BF, seed=1, behind=0)
    check(c, *run(c))
    c["max_nodes"] = 7
    check(c, *run(c), max_nodes=7)
    c["max_nodes"] = 20
    for T in (5, 14, 30):
        short = dict(c, q=c["q"][:T].contiguous(), bits=c["bits"][:T])
        check(short, *run(short))
    c["lengths"][1] = 10**6  # past the table's room: clipped
    c["lengths"][2] = -4
    check(c, *run(c))


@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("m", [4, 40])
@pytest.mark.parametrize("page", [16, 64, 6])
def test_what_no_key_holds_is_not_used(page, m, kind):
    """Places past a sequence's end, before its window and pages of nobody hold NaN and infinities; holes are
    passed over."""
    lengths, window = [m, 333, 90, 45], 200
    c = make(4, 2, 64, lengths, [m, m, 1, 2], page, BF, kind, seed=3)
    k, table = c["k"], c["table"]
    table[1, 2], table[1, 4], table[1, 5] = -1, k.shape[0], 2**31 - 1
    table[3, :] = -5
    live = torch.zeros(k.shape[:2], dtype=torch.bool)
    for b, n in enumerate(lengths):
        for j in range(max(0, n - m - window), n):
            p = int(table[b, j // page])
            if 0 <= p < k.shape[0]:
                live[p, j % page] = True
    ref = run(c, window=window)
    check(c, *ref, window=window)
    bad = ~live.to(DEV)
    for t in (c["k"], c["v"]):
        if kind == "e4m3":
            t.view(torch.uint8)[bad] = 0x7F
        else:
            t[bad] = math.nan
            t[bad.nonzero()[::2, 0], bad.nonzero()[::2, 1]] = math.inf
    got = run(c, window=window)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("m", [4, 40])
@pytest.mark.parametrize("page", [16, 3])
def test_a_branch_that_is_not_finite_stays_in_it(page, m, kind):
    """Keys and values of one node NaN or infinite: the rows that do not see it are as if it were zero."""
    c = make(8, 2, 80, [m + 70, m], [m, m], page, HF, kind, seed=4)
    b, node = 0, m // 2
    key = 70 + node
    at = int(c["table"][b, key // page]), key % page
    sees = torch.tensor([bool(x >> node & 1) for x in c["bits"][:m]] + [False] * (m + 3))
    assert sees.any() and not sees.all()
    for t, bad in ((c["k"], math.nan), (c["v"], math.nan), (c["v"], math.inf)):
        if bad == math.inf and kind == "e4m3":
            continue
        keep = t.clone()
        u = t.view(torch.uint8) if kind == "e4m3" else t
        u[at] = 0x00 if kind == "e4m3" else 0.0
        ref = run(c)
        u[at] = 0x7F if kind == "e4m3" else bad
        out, lse = run(c)
        tol = 2.0 ** -10  # the same sums in another order: a rounding of the result apart
        assert ((out - ref[0])[~sees].abs() <= tol * (1 + ref[0][~sees].abs())).all()
        assert torch.equal(lse[~sees], ref[1][~sees])
        if bad == math.inf:
            assert (out[sees] == math.inf).all() and torch.equal(lse[sees], ref[1][sees])
        else:
            assert torch.isnan(out[sees]).all()
        t.copy_(keep)


def test_views_and_in_place():
    """Heads of a fused projection as q, results onto it; a table's rows apart."""
    c = make(4, 2, 64, [70, 40], [5, 9], 16, BF, seed=5)
    ref = run(c)
    T = c["q"].shape[0]
    wide = torch.full((T, 3, 4, 64), 2.0, dtype=BF, device=DEV)
    wide[:, 1] = c["q"]
    table = torch.full((2, 20), -1, dtype=torch.int32, device=DEV)
    table[:, :c["table"].shape[1]] = c["table"]
    tree = tree_tensor(c["bits"], 1)
    out = tcm.paged_tree_attention(wide[:, 1], c["k"], c["v"], table[:, :c["table"].shape[1]], c["lengths"], c["starts"], 9,
                                   tree=tree, out=wide[:, 1])
    assert torch.equal(out[:14], ref[0][:14]) and torch.equal(out[14:], c["q"][14:])
    assert (wide[:, 0] == 2).all() and (wide[:, 2] == 2).all()


def test_one_token_is_paged_attention():
    """One new token per sequence: what paged_attention gives, within the rounding of the results.  Either is off
    by half a step and the sums' errors (2^-16 of the magnitudes, far below); so they may be a whole step apart,
    and a bf16 step is 2^-7 of the value just above a power of two."""
    c = make(16, 4, 128, [1, 333, 2000, 64], [1] * 4, 16, BF, seed=6, tree=False, behind=0)
    out, lse = run(c)
    ref = tcm.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lengths"])
    assert ((out.float() - ref.float()).abs() <= (2.0 ** -7 + 2.0 ** -12) * ref.float().abs() + 1e-6).all()


def test_probabilities_far_below_the_largest():
    """Thousands of keys 2^-24 below the largest, together a part of the result that fp16 shows."""
    n, D = 4097, 64
    k = torch.zeros((1, 4112, 1, D), dtype=HF, device=DEV)
    v = torch.zeros_like(k)
    k[0, 0, 0, 0] = 1.0
    v[0, 1:n, 0] = 4096.0
    q = torch.zeros((3, 1, D), dtype=HF, device=DEV)
    q[:, 0, 0] = 1.0
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    out = tcm.paged_tree_attention(q, k, v, i32(0).view(1, 1), i32(n), i32(0, 3), 3, scale=24 * math.log(2))
    p = 2.0 ** -24
    for t in range(3):
        rest = n - 3 + t
        want = 4096.0 * rest * p / (1 + rest * p)
        assert abs(float(out[t, 0, 0]) / want - 1) < 2.0 ** -10
