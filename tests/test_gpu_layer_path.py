"""The layer operators together: the example's layer against a float64 model of it, on other
streams, from several threads, and in a graph."""
import concurrent.futures as cf
import os
import sys

import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_layer  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_example_against_a_float64_model(cache):
    """Each step's output from the inputs that the kernels had: keys and values of all
    earlier steps recomputed in float64.  What is rounded between the operators is
    independent from element to element: bf16 three times (q; k or v; the attention's
    result) 2^-9 / sqrt(3) of the size each, E4M3 caches 2^-4 / sqrt(3) of keys and values
    on top, averaged over the keys; the bounds are on the relative 2-norm of a step."""
    steps, B = 40, 5
    layer = decode_layer.Layer(cache=cache, pages=B * 3)
    adapter = torch.tensor([b % 5 - 1 for b in range(B)], dtype=torch.int32, device=DEV)
    x = torch.randn((B, 1024), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    seen = decode_layer.decode(layer, x, adapter, steps)
    h, hk, d = layer.heads, layer.kv_heads, layer.head_dim
    rows, sc, f = adapter.tolist(), f64(layer.scales), f64(layer.inv_freq)
    ks, vs = [[] for _ in range(B)], [[] for _ in range(B)]
    for t, (xt, out) in enumerate(seen):
        qkv, _ = ol.lora(f64(xt), f64(layer.w_qkv), f64(layer.a_qkv), f64(layer.b_qkv), rows, sc)
        qkv = qkv.reshape(B, h + 2 * hk, d)
        att = np.zeros((B, h * d))
        for b in range(B):
            if t < b:
                continue
            q = ol.norm_rope(qkv[b:b + 1, :h], [t - b], f, f64(layer.wq))[0]
            ks[b].append(ol.norm_rope(qkv[b:b + 1, h:h + hk], [t - b], f, f64(layer.wk))[0])
            vs[b].append(qkv[b, h + hk:])
            k, v = np.array(ks[b]), np.array(vs[b])
            for i in range(h):
                s = k[:, i // (h // hk)] @ q[i] / np.sqrt(d)
                p = np.exp(s - s.max())
                att[b, i * d:(i + 1) * d] = p @ v[:, i // (h // hk)] / p.sum()
        ref, _ = ol.lora(att, f64(layer.w_out), f64(layer.a_out), f64(layer.b_out), rows, sc)
        err = np.linalg.norm(f64(out) - ref) / np.linalg.norm(ref)
        assert err < (0.015 if cache == "same" else 0.12), (t, err)
        assert (f64(out)[[b for b in range(B) if t < b]] == 0).all()  # no key yet


def layer_state(seed, T=24):
    layer = decode_layer.Layer(seed=seed, pages=32)
    g = torch.Generator().manual_seed(seed + 50)
    x = torch.randn((T, 1024), generator=g).to(torch.bfloat16).to(DEV)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    n = [1 + (7 * b) % 16 for b in range(T)]
    args = (i32([b % 5 - 1 for b in range(T)]), i32([m - 1 for m in n]), i32([16 * b + m - 1 for b, m in enumerate(n)]),
            i32([[b] for b in range(T)]), i32(n), 16)
    layer.k_cache.normal_()
    layer.v_cache.normal_()
    return layer, x, args


def test_on_a_side_stream_behind_other_work():
    """All calls go to the current stream: inputs written there just before, behind a spin,
    are seen, and a copy queued after sees the result."""
    layer, x, args = layer_state(1)
    want = layer.step(x, *args)
    torch.cuda.synchronize()
    late = torch.zeros_like(x)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        late.copy_(x)
        seen = layer.step(late, *args).clone()
    side.synchronize()
    assert torch.equal(seen, want)


def test_threads_on_their_own_streams():
    states = [layer_state(s) for s in range(4)]
    want = [layer.step(x, *args) for layer, x, args in states]
    torch.cuda.synchronize()

    def work(i):
        layer, x, args = states[i]
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            outs = [layer.step(x, *args) for _ in range(5)]
        st.synchronize()
        return outs

    with cf.ThreadPoolExecutor(4) as ex:
        for i, outs in enumerate(ex.map(work, range(4))):
            assert all(torch.equal(o, want[i]) for o in outs)


def test_in_a_graph():
    """A step and a backward pass captured once: replays, with eager work between them, give
    the eager bits, also after the inputs changed in place."""
    layer, x, args = layer_state(3)
    q, k = (torch.randn((700, n, 64), device=DEV).to(torch.bfloat16) for n in (8, 2))
    pos = torch.arange(700, dtype=torch.int32, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    long = [torch.randn((64, 16, 2, 64), device=DEV).to(torch.bfloat16) for _ in range(2)]
    table = torch.randperm(64, device=DEV).to(torch.int32).view(1, 64)
    n = torch.tensor([1000], dtype=torch.int32, device=DEV)

    def calls():
        return (layer.step(x, *args), *tcm.qk_norm_rope_bwd(q, k, q, k, pos, layer.inv_freq, w, w),
                tcm.paged_attention(q[:1], *long, table, n, max_len=1024))

    eager = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for r in range(3):
        for t in got:
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), r
    x.mul_(-0.5)
    q.mul_(2.0)
    n.fill_(300)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in got]
    for a, b in zip(replayed, calls()):
        assert torch.equal(a, b)
