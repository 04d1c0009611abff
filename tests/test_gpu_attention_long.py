"""Long sequences whose every part can be seen: the keys beside each place where a split may begin
or end have nearly all of the weight and values of their own, so that a key or a part that is
lost, taken twice or taken in another's place shows beyond the tolerance.  That it does is itself
tested, on the CPU, with such mistakes in the reference's place."""
import math

import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol
from test_gpu_attention_precision import close, f64

DEV = "cuda"
D = 16


def marks(n):
    """The first and last key, and both sides of every multiple of 1024 (of 256 below 40000 keys):
    chunks are 256, 384, .. 1024 keys."""
    step = 1024 if n > 40000 else 256
    edges = {0, n - 1}
    for m in range(step, n, step):
        edges |= {m - 1, m}
    return np.array(sorted(edges))


def planted(n, dtype, seed):
    """Keys (n, D), values (n, D) and a query (D,): marked keys score 8, others 0 and below."""
    g = np.random.default_rng(seed)
    k, v = 0.5 * g.normal(size=(n, D)), g.normal(size=(n, D))
    k[:, 0] = -np.abs(k[:, 0])
    at = marks(n)
    k[at, 0] = 8.0
    v[at] = g.choice([-1.0, 1.0], size=(len(at), D)) * g.integers(4, 17, size=(len(at), D)) / 8.0
    q = np.zeros(D)
    q[0] = 1.0
    q[1:] = 0.125
    rounded = lambda x: torch.from_numpy(x).to(dtype)  # noqa: E731
    return rounded(k), rounded(v), rounded(q)


def parts(k, v, q):
    """Weights of a row and its scores' sizes, in 64 bits."""
    s = k @ q
    e = np.exp(s - s.max())
    return s, e, (np.abs(k) @ np.abs(q)).max()


SIZES = [(1, 700), (1, 3000), (1, 5121), (1, 40001), (1, 65537), (1, 130049), (1, 131072), (2, 9000), (1, 261121)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", sorted({n for _, n in SIZES}))
def test_a_lost_part_would_be_seen(n, dtype):
    k, v, q = (f64(t) for t in planted(n, dtype, n))
    s, e, top = parts(k, v, q)
    ref, mag, rlse = e @ v / e.sum(), e @ np.abs(v) / e.sum(), s.max() + math.log(e.sum())

    def judge(weight, total):
        """What close() says of the output with these weights over this sum, rounded as the call's is."""
        out = torch.from_numpy(weight @ v / total).to(dtype).double().numpy()
        lse = np.array([[s.max() + math.log(total)]])
        close(out[None, None], None, ref[None, None], np.array([[rlse]]), mag[None, None], np.array([[top]]), dtype, D, n,
              np.abs(v).max())
        return lse

    judge(e, e.sum())
    chunk = 1024 if n > 40000 else 256
    last = (n - 1) // chunk
    wrong = {}
    for c in sorted({0, 1, last // 2, last - 1, last}):
        w = e.copy()
        w[c * chunk:(c + 1) * chunk] = 0
        wrong[f"chunk {c} lost"] = (w, w.sum())
        wrong[f"chunk {c} lost but for its sum"] = (w, e.sum())
        wrong[f"chunk {c} twice"] = (2 * e - w, (2 * e - w).sum())
    for key in (0, n - 1, chunk - 1, chunk, last * chunk):
        w = e.copy()
        w[key] = 0
        wrong[f"key {key} lost"] = (w, w.sum())
        wrong[f"key {key} twice"] = (2 * e - w, (2 * e - w).sum())
    for what, (w, total) in wrong.items():
        with pytest.raises(AssertionError):
            judge(w, total)
            pytest.fail(what)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hk", [1, 4, 8])
@pytest.mark.parametrize("B,n", SIZES)
def test_every_part_arrives(B, n, Hk, dtype):
    """Both ways to deal the keys out (a head a workgroup, four heads a workgroup), every head with keys
    of its own; the second sequence is one key shorter than a chunk's multiple."""
    page, per = 64, -(-n // 64)
    g = torch.Generator().manual_seed(n)
    table = torch.randperm(B * per, generator=g).view(B, per)
    kc, vc = (torch.zeros((B * per, page, Hk, D), dtype=dtype) for _ in range(2))
    lengths, q, want = [], torch.zeros((B, 2 * Hk, D), dtype=dtype), []
    for b in range(B):
        m = n if b == 0 else n // 1024 * 1024 - 1
        lengths.append(m)
        for h in range(Hk):
            k, v, one = planted(m, dtype, 31 * h + b)
            q[b, 2 * h], q[b, 2 * h + 1] = one, one * 0.5
            for cache, t in ((kc, k), (vc, v)):
                whole = torch.zeros((per * page, D), dtype=dtype)
                whole[:m] = t
                cache[table[b], :, h] = whole.view(per, page, D)
            for i in (0, 1):
                s, e, top = parts(f64(k), f64(v), f64(q[b, 2 * h + i]))
                want.append((e @ f64(v) / e.sum(), s.max() + math.log(e.sum()), e @ np.abs(f64(v)) / e.sum(), top))
    lse = torch.full((B, 2 * Hk), math.nan, dtype=torch.float32, device=DEV)
    out = tcm.paged_attention(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(torch.int32).to(DEV),
                              torch.tensor(lengths, dtype=torch.int32, device=DEV), scale=1.0, lse=lse)
    ref, rlse, mag, top = (np.array([w[i] for w in want]).reshape((B, 2 * Hk) + ((D,) if i in (0, 2) else ()))
                           for i in range(4))
    close(f64(out), f64(lse), ref, rlse, mag, top, dtype, D, n, 4.0)
