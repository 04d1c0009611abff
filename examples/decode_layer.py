"""One attention layer of a server, token by token, for several requests at once.

Every request has an adapter of its own (or none) beside the shared projections, a list
of pages in one shared cache, and a length of its own.  A step takes one new token of
every request:

    qkv   = x W_qkv^T + its adapter            lora_gemm_tn
    q, k  = norm and rotation; k, v -> cache   qk_norm_rope_cache
    a     = attention over its pages           paged_attention
    out   = a W_out^T + its adapter            lora_gemm_tn

    python examples/decode_layer.py [--requests 8] [--steps 40] [--cache e4m3]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tensor_core_matrix_amd as tcm  # noqa: E402


class Layer:
    """Weights, adapters and a paged cache of one attention layer."""

    def __init__(self, width=1024, heads=16, kv_heads=4, head_dim=64, adapters=4, rank=16, pages=256,
                 page_size=16, cache="same", dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s, sd=1.0: (torch.randn(s, generator=g) * sd).to(dtype).to(device)  # noqa: E731
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.page_size, self.free = page_size, list(range(pages))
        nq, nkv = heads * head_dim, kv_heads * head_dim
        self.w_qkv = n(nq + 2 * nkv, width, sd=width ** -0.5)
        self.w_out = n(width, nq, sd=nq ** -0.5)
        self.a_qkv = n(adapters, rank, width, sd=width ** -0.5)
        self.b_qkv = n(adapters, nq + 2 * nkv, rank, sd=0.3 * rank ** -0.5)
        self.a_out = n(adapters, rank, nq, sd=nq ** -0.5)
        self.b_out = n(adapters, width, rank, sd=0.3 * rank ** -0.5)
        self.scales = torch.full((adapters,), 2.0, device=device)
        self.wq, self.wk = 1 + n(head_dim, sd=0.1), 1 + n(head_dim, sd=0.1)
        self.inv_freq, self.factor = tcm.rope_frequencies(head_dim, device=device)
        kind = torch.float8_e4m3fn if cache == "e4m3" else dtype
        shape = (pages, page_size, kv_heads, head_dim)
        self.k_cache = torch.empty(shape, dtype=kind, device=device)
        self.v_cache = torch.empty(shape, dtype=kind, device=device)
        self.k_scale, self.v_scale = (1 / 32, 1 / 64) if cache == "e4m3" else (1.0, 1.0)

    def step(self, x, adapter, positions, slots, table, lengths, max_len):
        """The layer's output for one token of every request: x (requests, width), its
        adapter numbers, the tokens' positions and cache slots, and the sequences' pages and
        lengths with these tokens."""
        d, h, hk = self.head_dim, self.heads, self.kv_heads
        qkv = tcm.lora_gemm_tn(x, self.w_qkv, self.a_qkv, self.b_qkv, adapter, scales=self.scales)
        q, k, v = qkv.view(-1, h + 2 * hk, d).split([h, hk, hk], 1)
        q = tcm.qk_norm_rope_cache(q, k, v, positions, self.inv_freq, self.k_cache, self.v_cache, slots, self.wq,
                                   self.wk, factor=self.factor, k_scale=self.k_scale, v_scale=self.v_scale)
        a = tcm.paged_attention(q, self.k_cache, self.v_cache, table, lengths, max_len=max_len,
                                k_scale=self.k_scale, v_scale=self.v_scale, out=q)
        return tcm.lora_gemm_tn(a.view(-1, h * d), self.w_out, self.a_out, self.b_out, adapter, scales=self.scales)


def decode(layer, x, adapter, steps):
    """`steps` steps of every request from an empty cache, a step's output (scaled to unit
    size) being the next one's input; request b begins b steps after the first and only
    pads the batch until then.  Returns the inputs and outputs of every step."""
    B, device = x.shape[0], x.device
    per = -(-steps // layer.page_size)
    table = torch.full((B, per), -1, dtype=torch.int32, device=device)
    seen = []
    for t in range(steps):
        length = [max(0, t + 1 - b) for b in range(B)]
        slots = []
        for b, n in enumerate(length):
            if n and (n - 1) % layer.page_size == 0:
                table[b, (n - 1) // layer.page_size] = layer.free.pop()
        pages = table.tolist()
        for b, n in enumerate(length):
            j = n - 1
            slots.append(pages[b][j // layer.page_size] * layer.page_size + j % layer.page_size if n else -1)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
        out = layer.step(x, adapter, i32([max(0, n - 1) for n in length]), i32(slots), table, i32(length), steps)
        seen.append((x, out))
        x = (out.float() / out.float().square().mean(1, keepdim=True).add(1e-6).sqrt()).to(out.dtype)
    return seen


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--cache", choices=["same", "e4m3"], default="same")
    a = ap.parse_args()
    layer = Layer(cache=a.cache, pages=a.requests * (a.steps // 16 + 1))
    x = torch.randn((a.requests, 1024), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    adapter = torch.tensor([b % 5 - 1 for b in range(a.requests)], dtype=torch.int32, device="cuda")
    t = time.perf_counter()
    seen = decode(layer, x, adapter, a.steps)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.requests} requests x {a.steps} tokens, {a.cache} cache: {1e6 * t / a.steps:.0f} us a step, "
          f"last outputs {seen[-1][1].float().square().mean().sqrt().item():.4f} rms")


if __name__ == "__main__":
    main()
