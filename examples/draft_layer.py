"""One layer of a server whose requests draft several tokens a step and keep those that are right.

Weights have 4 bits (the products have few rows), the wide projection takes MXFP8 of both sides.
A step takes a small tree of drafted tokens of every request: a main branch, and a side
branch that begins at the main branch's first token.

    pages for the new tokens, their slots and positions     cache_plan
    x, residual -> residual + x, its norm                   add_rms_norm
    qkv = y W_qkv^T                                         gemm_w4
    q, k = norm and rotation; k, v -> cache                 qk_norm_rope_cache
    a   = attention over the pages, drafts by their tree    paged_tree_attention
    o   = a W_out^T                                         gemm_w4
    residual + o, its norm in MXFP8                         add_rms_norm_mx_fp8
    u   = z W_up^T                                          gemm_mx_fp8
    x   = (silu(u_1) u_2) W_down^T                          gemm_w4 (E2M1)
    pages of the drafts that were refused go back           cache_plan

    python examples/draft_layer.py [--requests 8] [--steps 20]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tensor_core_matrix_amd as tcm  # noqa: E402


class Layer:
    """Weights and a paged cache of one layer."""

    def __init__(self, width=1024, heads=16, kv_heads=4, head_dim=64, hidden=1280, group=64, pages=256, page_size=16,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s, sd=1.0: (torch.randn(s, generator=g) * sd).to(dtype).to(device)  # noqa: E731
        byte = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g).to(torch.uint8).to(device)  # noqa: E731

        def u4(N, K):  # weights of about 1 / sqrt(K): (q - zero) has 4.6 rms
            scales = ((0.8 + 0.4 * torch.rand((N, K // group), generator=g)) / 4.7 * K ** -0.5).to(dtype).to(device)
            return byte(0, 256, N, K // 2), scales, byte(6, 10, N, K // group)

        self.heads, self.kv_heads, self.head_dim, self.page_size = heads, kv_heads, head_dim, page_size
        nq, nkv = heads * head_dim, kv_heads * head_dim
        self.norm1, self.norm2 = 1 + n(width, sd=0.1), 1 + n(width, sd=0.1)
        self.w_qkv, self.w_out = u4(nq + 2 * nkv, width), u4(width, nq)
        self.w_up = n(2 * hidden, width, sd=16.0).to(torch.float8_e4m3fn)
        self.up_scale = byte(117, 119, 2 * hidden, width // 32)  # 2^-10, 2^-9
        self.w_down = byte(0, 256, width, hidden // 2)
        self.down_scale = byte(119, 121, width, hidden // 32)
        self.wq, self.wk = 1 + n(head_dim, sd=0.1), 1 + n(head_dim, sd=0.1)
        self.inv_freq, self.factor = tcm.rope_frequencies(head_dim, device=device)
        self.k_cache, self.v_cache = (torch.zeros((pages, page_size, kv_heads, head_dim), dtype=dtype, device=device)
                                      for _ in range(2))
        # the stack of free pages
        self.free_pages = torch.arange(pages, dtype=torch.int32, device=device)
        self.free_count = torch.tensor([pages], dtype=torch.int32, device=device)

    def plan(self, lengths, change, table, tokens):
        return tcm.cache_plan(lengths, change, table, self.free_pages, self.free_count, self.page_size, tokens=tokens)

    def step(self, x, residual, slots, positions, table, lengths, starts, nodes, tree, max_len):
        """(x, residual) of the next layer for the new tokens (rows) of all requests."""
        d, h, hk = self.head_dim, self.heads, self.kv_heads
        y, residual = tcm.add_rms_norm(x, self.norm1, residual=residual)
        qkv = tcm.gemm_w4(y, *self.w_qkv)
        q, k, v = qkv.view(-1, h + 2 * hk, d).split([h, hk, hk], 1)
        q = tcm.qk_norm_rope_cache(q, k, v, positions, self.inv_freq, self.k_cache, self.v_cache, slots, self.wq,
                                   self.wk, factor=self.factor)
        a = torch.zeros_like(q)  # (rows of no request stay as they are)
        tcm.paged_tree_attention(q, self.k_cache, self.v_cache, table, lengths, starts, nodes, tree=tree,
                                 max_len=max_len, out=a)
        o = tcm.gemm_w4(a.view(-1, h * d), *self.w_out)
        z, zs, residual = tcm.add_rms_norm_mx_fp8(o, self.norm2, residual=residual)
        one, two = tcm.gemm_mx_fp8(z, self.w_up, zs, self.up_scale, out_dtype=torch.bfloat16).chunk(2, 1)
        act = (torch.nn.functional.silu(one.float()) * two.float()).to(x.dtype)
        return tcm.gemm_w4(act, self.w_down, self.down_scale, elem="e2m1"), residual


def branches(main, side):
    """For main + side nodes of a request: the bits of what each sees, and how much less its
    position is than its place behind the context."""
    bits, less = [], []
    for i in range(main + side):
        below = range(i + 1) if i < main else [0, *range(main, i + 1)]
        bits.append(sum(1 << j for j in below))
        less.append(0 if i < main else main - 1)
    return bits, less


def decode(layer, requests, steps, main=4, side=3, seed=1, seen=None):
    """`steps` steps of drafts; of each request's main branch a random part is kept (at least the
    first token).  Every fourth request begins later and has no tokens until then.  Returns the lengths."""
    g = torch.Generator().manual_seed(seed)
    nodes, device = main + side, layer.k_cache.device
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
    most = steps * main + nodes
    lengths = torch.zeros(requests, dtype=torch.int32, device=device)
    table = torch.full((requests, -(-most // layer.page_size)), -1, dtype=torch.int32, device=device)
    bits, less = branches(main, side)
    T = requests * nodes
    for t in range(steps):
        active = [b for b in range(requests) if b % 4 != 3 or t >= 3]
        new = [nodes if b in active else 0 for b in range(requests)]
        pad = T - len(active) * nodes  # rows behind the last request's
        tree = torch.tensor(bits * len(active) + [0] * pad, device=device).view(T, 1)
        starts, slots, positions = layer.plan(lengths, i32(new), table, T)
        positions -= i32(less * len(active) + [0] * pad)
        x, residual = (torch.randn((T, layer.norm1.numel()), generator=g).to(layer.norm1.dtype).to(device) for _ in range(2))
        out = layer.step(x, residual, slots, positions, table, lengths, starts, nodes, tree, most)
        kept = [1 + int(torch.randint(0, main, (), generator=g)) if n else 0 for n in new]
        if seen is not None:
            seen.append((x, residual, *out, active, kept))
        layer.plan(lengths, i32([k - n for k, n in zip(kept, new)]), table, 0)
    return lengths


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    layer = Layer(pages=a.requests * (a.steps // 4 + 2))
    t = time.perf_counter()
    lengths = decode(layer, a.requests, a.steps)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.requests} requests, {a.steps} steps: {int(lengths.sum())} tokens kept, {1e6 * t / a.steps:.0f} us a step, "
          f"{int(layer.free_count)} of {len(layer.free_pages)} pages free")


if __name__ == "__main__":
    main()
