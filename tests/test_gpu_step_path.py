"""The operators of a step that drafts together: the example's layer against a float64 model of it,
on other streams, from several threads, and in a graph with what takes and returns the pages."""
import concurrent.futures as cf
import os
import sys

import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol
from oracle import step as os_

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import draft_layer  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.double().cpu().numpy()


def w4(x, w, elem="u4"):
    """x times the weights of gemm_w4 as the layer holds them"""
    packed, scales, zeros = w if len(w) == 3 else (*w, None)
    scales = scales.cpu().numpy() if elem == "e2m1" else f64(scales)
    return os_.gemm_w4(x, packed.cpu().numpy(), scales, None if zeros is None else zeros.cpu().numpy(), elem)[0]


def test_example_against_a_float64_model():
    """Each step's results from the inputs that the kernels had, keys and values of all kept tokens
    recomputed in float64.  A rounding to bf16 is 2^-9 of a value at most on the way to the
    residual (2^-9 / sqrt(3) rms): y, qkv, q, k, v, the attention's result, o and the residual itself, eight
    independent ones, sqrt(8 / 3) 2^-9 = 0.0032 of the result; 0.015 is allowed as for the layer without drafts.
    The elements of z have 2^-4 / sqrt(3) rms at most, which two factors of the product behind
    have: sqrt(2) 0.036 = 0.051, and 0.12 is allowed."""
    B, steps, mainb, side = 5, 9, 4, 3
    nodes = mainb + side
    layer = draft_layer.Layer(pages=24)
    seen = []
    lengths = draft_layer.decode(layer, B, steps, mainb, side, seen=seen)
    h, hk, d = layer.heads, layer.kv_heads, layer.head_dim
    f, bits = f64(layer.inv_freq), draft_layer.branches(mainb, side)[0]
    ks, vs = [[] for _ in range(B)], [[] for _ in range(B)]
    up = f64(layer.w_up.to(torch.float32)) * np.repeat(2.0 ** (layer.up_scale.cpu().numpy().astype(float) - 127), 32, 1)
    for x, residual, out, kept_residual, active, kept in seen:
        y, s1 = os_.add_rms_norm(f64(x), f64(residual), f64(layer.norm1))
        qkv = w4(y, layer.w_qkv).reshape(-1, h + 2 * hk, d)
        att = np.zeros((len(x), h * d))
        for i, b in enumerate(active):
            rows = slice(i * nodes, (i + 1) * nodes)
            context = len(ks[b])
            pos = [context + bin(w).count("1") - 1 for w in bits]
            q = ol.norm_rope(qkv[rows, :h], pos, f, f64(layer.wq))
            new_k, new_v = ol.norm_rope(qkv[rows, h:h + hk], pos, f, f64(layer.wk)), qkv[rows, h + hk:]
            k, v = np.array(ks[b] + list(new_k)), np.array(vs[b] + list(new_v))
            for j in range(nodes):
                see = [*range(context), *(context + n for n in range(nodes) if bits[j] >> n & 1)]
                for c in range(h):
                    s = k[see, c // (h // hk)] @ q[j, c] / np.sqrt(d)
                    p = np.exp(s - s.max())
                    att[i * nodes + j, c * d:(c + 1) * d] = p @ v[see, c // (h // hk)] / p.sum()
            ks[b] += list(new_k[:kept[b]])
            vs[b] += list(new_v[:kept[b]])
        z, s2 = os_.add_rms_norm(w4(att, layer.w_out), s1, f64(layer.norm2))
        one, two = np.split(z @ up.T, 2, 1)
        ref = w4(one / (1 + np.exp(-one)) * two, (layer.w_down, layer.down_scale), "e2m1")
        for got, want, most in ((kept_residual, s2, 0.015), (out, ref, 0.12)):
            assert np.linalg.norm(f64(got) - want) < most * np.linalg.norm(want)
    assert lengths.tolist() == [len(k) for k in ks]
    used = sum(-(-len(k) // layer.page_size) for k in ks)
    assert int(layer.free_count) == 24 - used
    assert len(set(layer.free_pages[:24 - used].tolist())) == 24 - used


class State:
    """A step of drafts that begins and ends with the same lengths and pages."""

    def __init__(self, seed, B=6, main=4, side=3, most=200):
        g = torch.Generator().manual_seed(seed + 50)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        self.layer = draft_layer.Layer(seed=seed, pages=120)
        self.layer.k_cache.normal_()
        self.layer.v_cache.normal_()
        self.nodes, self.most, self.T = main + side, most, B * (main + side) + 5
        bits, less = draft_layer.branches(main, side)
        self.tree = torch.tensor(bits * B + [0] * 5, device=DEV).view(-1, 1)
        self.less = i32(less * B + [0] * 5)
        self.lengths = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.table = torch.full((B, 13), -1, dtype=torch.int32, device=DEV)
        self.layer.plan(self.lengths, i32([7 + 29 * b for b in range(B)]), self.table, 0)
        self.more = torch.full((B,), self.nodes, dtype=torch.int32, device=DEV)
        self.back = -self.more
        self.x, self.residual = (torch.randn((self.T, 1024), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))

    def step(self, x=None):
        starts, slots, positions = self.layer.plan(self.lengths, self.more, self.table, self.T)
        out = self.layer.step(self.x if x is None else x, self.residual, slots, positions - self.less, self.table,
                              self.lengths, starts, self.nodes, self.tree, self.most)
        self.layer.plan(self.lengths, self.back, self.table, 0)
        return (*out, slots, starts)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_on_a_side_stream_behind_other_work():
    st = State(1)
    want = [t.clone() for t in st.step()]
    torch.cuda.synchronize()
    late = torch.zeros_like(st.x)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        late.copy_(st.x)
        seen = [t.clone() for t in st.step(late)]
    side.synchronize()
    assert same(seen, want)


def test_threads_on_their_own_streams():
    states = [State(s) for s in range(4)]
    want = [st.step() for st in states]
    torch.cuda.synchronize()

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            outs = [states[i].step() for _ in range(5)]
        stream.synchronize()
        return outs

    with cf.ThreadPoolExecutor(4) as ex:
        for i, outs in enumerate(ex.map(work, range(4))):
            assert all(same(o, want[i]) for o in outs)


def test_in_a_graph():
    """The step and a gradient captured once: replays, with eager work between them, give the eager bits,
    also after the inputs and the lengths changed in place."""
    st = State(3)
    w = st.layer.norm1.float()

    def calls():
        out = st.step()
        return (*out, *tcm.add_rms_norm_bwd(st.x, st.residual, w, dsum=st.x))

    eager = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    state = [t.clone() for t in (st.lengths, st.table, st.layer.free_pages, st.layer.free_count)]
    for r in range(3):
        for t in got:
            t.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, eager), r
        assert same((st.lengths, st.table, st.layer.free_pages, st.layer.free_count), state)
    st.x.mul_(-0.5)
    st.layer.plan(st.lengths, torch.tensor([9, -20, 0, 3, -94, 17], dtype=torch.int32, device=DEV), st.table, 0)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in got]
    assert same(replayed, calls())


def test_two_graphs_with_a_workspace_each_share_nothing():
    """Captured calls with workspaces of their own, replayed on two streams at once."""
    q, k, v = (torch.randn(s, device=DEV).to(torch.bfloat16) for s in ((6, 8, 64), (64, 16, 2, 64), (64, 16, 2, 64)))
    table = torch.randperm(64, device=DEV).to(torch.int32).view(2, 32)
    n, starts = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([500, 321], [0, 4, 6]))
    bytes_ = tcm.paged_tree_attention_workspace(2, 8, 2, 64, 4, 512)
    want = tcm.paged_tree_attention(q, k, v, table, n, starts, 4, max_len=512).clone()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        ws, out = torch.empty(bytes_, dtype=torch.uint8, device=DEV), torch.empty_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tcm.paged_tree_attention(q, k, v, table, n, starts, 4, max_len=512, out=out, workspace=ws)
        graphs.append((graph, torch.cuda.Stream(), out))
    for _ in range(5):
        for graph, stream, out in graphs:
            out.zero_()
        torch.cuda.synchronize()
        for graph, stream, out in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, _, out in graphs)
