"""Cases of the operators of one attention layer in a server: the projection with low-rank adapters, the
norms and rotation of queries and keys (into a paged cache, and backwards), and the attention of one new
token over that cache.

`run` computes them in their plain form (elementary torch operations in 32 bits, rounded once) or, with
`own`, through the library's entry points.  `exact` computes them from their definitions in 64 bits.

    lora        Out[i] = X[i] W^T + s_a (X[i] A_a^T) B_a^T, a the adapter of row i (-1: none)
    rope        n = x w / sqrt(mean(x^2) + eps) per head; the first `rot` elements rotated by
                position * inv_freq; q dense, k and v into the pages of a cache (slot -1: nothing written)
    rope_bwd    gradients of q, k and the two norm weights of the same without a cache
    attention   o = softmax(scale q k^T) v over the last `window` keys (0: all) of a sequence's pages
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
K_SCALE, V_SCALE = 0.0625, 0.03125  # what a value of 1 in an 8-bit cache of keys, of values, stands for


def listed():
    return [
        # one token of one request through a 4096 x 4096 projection: latency
        dict(name="lora_m1", op="lora", M=1, N=4096, K=4096, R=16, L=8, dtype="bf16", out="bf16", mix="rows"),
        # a decode batch, nearly every row with an adapter of its own
        dict(name="lora_m48", op="lora", M=48, N=8192, K=4096, R=32, L=64, dtype="f16", out="f16", mix="rows"),
        # prompts of several requests, packed: odd number of rows, few adapters a tile
        dict(name="lora_m333", op="lora", M=333, N=4096, K=4096, R=8, L=16, dtype="bf16", out="f32", mix="runs"),
        # long prompts packed to 4096 rows: bound by the matrix cores
        dict(name="lora_m4096", op="lora", M=4096, N=4096, K=4096, R=16, L=16, dtype="bf16", out="bf16", mix="runs"),
        # a decode step's new tokens into the cache
        dict(name="rope_t64", op="rope", T=64, Hq=32, Hk=8, D=128, rot=128, page=16, layout="half", dtype="bf16",
             cache="same", start=100000),
        # a long prompt into an 8-bit cache: bound by memory
        dict(name="rope_t8191", op="rope", T=8191, Hq=32, Hk=8, D=128, rot=128, page=64, layout="half",
             dtype="bf16", cache="e4m3", start=0),
        # training, short: interleaved pairs on part of the head
        dict(name="rope_bwd_t512", op="rope_bwd", T=512, Hq=16, Hk=4, D=64, rot=32, layout="interleaved",
             dtype="f16", start=0),
        # training, a whole batch of tokens
        dict(name="rope_bwd_t8192", op="rope_bwd", T=8192, Hq=32, Hk=8, D=128, rot=128, layout="half",
             dtype="bf16", start=0),
        # one request that has just begun: latency
        dict(name="attn_b1_short", op="attention", B=1, Hq=32, Hk=8, D=128, most=200, page=16, dtype="bf16",
             cache="same", window=0),
        # a decode batch of ragged lengths
        dict(name="attn_b64", op="attention", B=64, Hq=32, Hk=8, D=128, most=4096, page=16, dtype="bf16",
             cache="same", window=0),
        # one request with a long context: split over its length
        dict(name="attn_b1_long", op="attention", B=1, Hq=32, Hk=8, D=128, most=131001, page=64, dtype="f16",
             cache="same", window=0),
        # a decode batch over an 8-bit cache
        dict(name="attn_b32_e4m3", op="attention", B=32, Hq=64, Hk=8, D=128, most=8192, page=64, dtype="bf16",
             cache="e4m3", window=0),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm (3072 apart)."""
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["lora", "rope", "rope_bwd", "attention"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "lora":
        eights = lambda: 8 * rng.choice([n for n in range(64, 513) if n != 384])  # noqa: E731
        return dict(op=op, M=_log(rng, 1, 4096), N=eights(), K=eights(), R=rng.choice([8, 16, 24, 32, 64]),
                    L=_log(rng, 1, 64), dtype=dtype, out=rng.choice([dtype, "f32"]), mix=rng.choice(["rows", "runs"]))
    D = rng.choice([64, 80, 96, 128, 128])
    Hk = rng.choice([1, 2, 4, 8])
    if op == "attention":
        B = _log(rng, 1, 64)
        Hq = Hk * rng.choice([1, 2, 4, 8])
        most = _log(rng, 1, min(131001, (1 << 21) // (B * Hk)))
        return dict(op=op, B=B, Hq=Hq, Hk=Hk, D=D, most=most, page=rng.choice([8, 16, 64, 128]), dtype=dtype,
                    cache=rng.choice(["same", "e4m3"]), window=rng.choice([0, 0, max(1, most // 3)]))
    c = dict(op=op, T=_log(rng, 1, 8192), Hq=Hk * rng.choice([1, 2, 4]), Hk=Hk, D=D,
             rot=rng.choice([D, D // 2, 32]), layout=rng.choice(["half", "interleaved"]), dtype=dtype,
             start=rng.choice([0, 1000, 500000]))
    if op == "rope":
        c.update(page=rng.choice([8, 16, 64]), cache=rng.choice(["same", "e4m3"]))
    return c


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, sigma, dt):
    return (torch.randn(shape, generator=g, device=DEV) * sigma).to(dt)


def _cache(shape, g, kind, dt, sigma):
    """Keys or values already in a cache; 8-bit ones as bytes."""
    if kind == "e4m3":
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16) * 16.0
        return x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float16) * sigma).to(dt)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    dt = DT[c["dtype"]]
    s = dict(c=c)
    if c["op"] == "lora":
        M, N, K, R, L = c["M"], c["N"], c["K"], c["R"], c["L"]
        s["x"] = _normal((M, K), g, 1.0, dt)
        s["w"] = _normal((N, K), g, K ** -0.5, dt)
        s["a"] = _normal((L, R, K), g, K ** -0.5, dt)
        s["b"] = _normal((L, N, R), g, 0.5 * R ** -0.5, dt)
        s["scales"] = 0.5 + torch.rand((L,), generator=g, device=DEV)
        if c["mix"] == "rows":  # a request a row
            rows = torch.randint(-1, L, (M,), generator=g, device=DEV)
        else:  # requests of consecutive rows
            n = max(1, min(M, L) // 2)
            of = torch.randint(-1, L, (n,), generator=g, device=DEV)
            ends = torch.sort(torch.randint(0, M + 1, (n - 1,), generator=g, device=DEV))[0]
            rows = of[torch.searchsorted(ends, torch.arange(M, device=DEV), right=True)]
        s["rows"] = rows.to(torch.int32)
        s["out"] = torch.empty((M, N), dtype=DT[c["out"]], device=DEV)
        if own:
            import tensor_core_matrix_amd as tcm
            s["ws"] = torch.empty(tcm.lora_workspace(M, K, R), dtype=torch.uint8, device=DEV)
        return s
    if c["op"] in ("rope", "rope_bwd"):
        T, Hq, Hk, D, rot = c["T"], c["Hq"], c["Hk"], c["D"], c["rot"]
        s["qkv"] = _normal((T, (Hq + 2 * Hk) * D), g, 1.0, dt)  # what a fused projection gives
        s["wq"] = (1 + 0.1 * torch.randn((D,), generator=g, device=DEV)).to(dt)
        s["wk"] = (1 + 0.1 * torch.randn((D,), generator=g, device=DEV)).to(dt)
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        s["pos"] = (c["start"] + torch.arange(T, device=DEV)).to(torch.int32)
        s["dq"] = torch.empty((T, Hq, D), dtype=dt, device=DEV)
        if c["op"] == "rope":
            pages = -(-2 * T // c["page"]) + 1
            s["kc"] = _cache((pages, c["page"], Hk, D), g, c["cache"], dt, 1.0)
            s["vc"] = _cache((pages, c["page"], Hk, D), g, c["cache"], dt, 1.0)
            slots = torch.randperm(pages * c["page"], generator=g, device=DEV)[:T]
            slots[torch.rand((T,), generator=g, device=DEV) < 0.02] = -1  # tokens that only pad the batch
            s["slots"] = slots.to(torch.int32)
        else:
            s["gq"] = _normal((T, Hq, D), g, 1.0, dt)
            s["gk"] = _normal((T, Hk, D), g, 1.0, dt)
            s["dk"] = torch.empty((T, Hk, D), dtype=dt, device=DEV)
            s["dw"] = torch.empty((2, D), dtype=torch.float32, device=DEV)
            if own:
                import tensor_core_matrix_amd as tcm
                s["ws"] = torch.empty(tcm.qk_norm_rope_bwd_workspace(D), dtype=torch.uint8, device=DEV)
        return s
    B, Hq, Hk, D, most, page = c["B"], c["Hq"], c["Hk"], c["D"], c["most"], c["page"]
    per = -(-most // page)
    pages = B * per
    s["q"] = _normal((B, Hq, D), g, 1.0, dt)
    s["kc"] = _cache((pages, page, Hk, D), g, c["cache"], dt, 1.0)
    s["vc"] = _cache((pages, page, Hk, D), g, c["cache"], dt, 1.0)
    lengths = torch.randint(1, most + 1, (B,), generator=g, device=DEV)
    lengths[0] = most
    if B > 2:
        lengths[1] = 0  # a slot of the batch without a request
    s["lengths"] = lengths.to(torch.int32)
    table = torch.randperm(pages, generator=g, device=DEV).view(B, per)
    used = torch.arange(per, device=DEV)[None, :] * page < lengths[:, None]
    s["table"] = torch.where(used, table, -1).to(torch.int32).contiguous()
    s["out"] = torch.empty((B, Hq, D), dtype=dt, device=DEV)
    s["lse"] = torch.empty((B, Hq), dtype=torch.float32, device=DEV)
    s["ks"], s["vs"] = (K_SCALE, V_SCALE) if c["cache"] == "e4m3" else (1.0, 1.0)
    if own:
        import tensor_core_matrix_amd as tcm
        s["ws"] = torch.empty(tcm.paged_attention_workspace(B, Hq, Hk, D, most), dtype=torch.uint8, device=DEV)
    return s


def _heads(s):
    """q, k and v of the fused projection's output, as views."""
    c = s["c"]
    Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
    x = s["qkv"].view(c["T"], Hq + 2 * Hk, D)
    return x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]


# ---- the library's entry points -------------------------------------------------------------------------

def _own(s):
    import tensor_core_matrix_amd as tcm
    c = s["c"]
    if c["op"] == "lora":
        tcm.lora_gemm_tn(s["x"], s["w"], s["a"], s["b"], s["rows"], scales=s["scales"], out=s["out"],
                         workspace=s["ws"])
        return {"out": s["out"]}
    if c["op"] == "rope":
        q, k, v = _heads(s)
        e4m3 = c["cache"] == "e4m3"
        tcm.qk_norm_rope_cache(q, k, v, s["pos"], s["inv_freq"], s["kc"], s["vc"], s["slots"], s["wq"], s["wk"],
                               eps=EPS, layout=c["layout"], k_scale=K_SCALE if e4m3 else 1.0,
                               v_scale=V_SCALE if e4m3 else 1.0, q_out=s["dq"])
        return {"q": s["dq"], "k_cache": s["kc"], "v_cache": s["vc"]}
    if c["op"] == "rope_bwd":
        q, k, _ = _heads(s)
        tcm.qk_norm_rope_bwd(s["gq"], s["gk"], q, k, s["pos"], s["inv_freq"], s["wq"], s["wk"], eps=EPS,
                             layout=c["layout"], dq=s["dq"], dk=s["dk"], dwq=s["dw"][0], dwk=s["dw"][1],
                             workspace=s["ws"])
        return {"dq": s["dq"], "dk": s["dk"], "dwq": s["dw"][0], "dwk": s["dw"][1]}
    tcm.paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["lengths"], window=c["window"], max_len=c["most"],
                        k_scale=s["ks"], v_scale=s["vs"], out=s["out"], lse=s["lse"], workspace=s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


# ---- the plain forms ------------------------------------------------------------------------------------

def _plain_lora(s):
    c = s["c"]
    M, N, L, R = c["M"], c["N"], c["L"], c["R"]
    x = s["x"].float()
    rows = s["rows"].long()
    mine = (rows[:, None] == torch.arange(L, device=DEV)[None, :]).float() * s["scales"][None, :]
    t = (x @ s["a"].float().view(L * R, -1).t()).view(M, L, R) * mine[:, :, None]
    y = x @ s["w"].float().t()
    y += t.view(M, L * R) @ s["b"].float().permute(0, 2, 1).reshape(L * R, N)
    return {"out": y.to(DT[c["out"]])}


def _cos_sin(s):
    # the angle in 64 bits, as its frequencies are given: a position of 2^19 leaves 32 bits no digit to lose
    t = s["pos"].double()[:, None] * s["inv_freq"][None, :]
    return t.cos().float()[:, None, :], t.sin().float()[:, None, :]


def _split(x, c):
    """The two elements of every rotated pair, and what is not rotated."""
    rot = c["rot"]
    a, rest = x[..., :rot], x[..., rot:]
    if c["layout"] == "half":
        return a[..., :rot // 2], a[..., rot // 2:], rest
    return a[..., 0::2], a[..., 1::2], rest


def _join(x1, x2, rest, c):
    pair = torch.cat((x1, x2), -1) if c["layout"] == "half" else torch.stack((x1, x2), -1).flatten(-2)
    return torch.cat((pair, rest), -1)


def _norm_rope(x, w, cos, sin, c):
    x = x.float()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    n1, n2, rest = _split(n, c)
    return _join(n1 * cos - n2 * sin, n2 * cos + n1 * sin, rest, c)


def _into(cache, slots, x, scale, c):
    keep = slots >= 0
    at = slots[keep].long()
    flat = cache.view(-1, c["Hk"], c["D"])
    if c["cache"] == "e4m3":
        flat.view(torch.uint8)[at] = (x[keep] / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        flat[at] = x[keep].to(cache.dtype)


def _plain_rope(s):
    c = s["c"]
    q, k, v = _heads(s)
    cos, sin = _cos_sin(s)
    _into(s["kc"], s["slots"], _norm_rope(k, s["wk"], cos, sin, c), K_SCALE, c)
    _into(s["vc"], s["slots"], v.float(), V_SCALE, c)
    return {"q": _norm_rope(q, s["wq"], cos, sin, c).to(q.dtype), "k_cache": s["kc"], "v_cache": s["vc"]}


def _norm_rope_grad(dy, x, w, cos, sin, c):
    x, dy = x.float(), dy.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    h = x * r
    y1, y2, rest = _split(dy, c)
    dn = _join(y1 * cos + y2 * sin, y2 * cos - y1 * sin, rest, c)
    g = dn * w.float()
    return r * (g - h * (g * h).mean(-1, keepdim=True)), (dn * h).sum((0, 1))


def _plain_rope_bwd(s):
    c = s["c"]
    q, k, _ = _heads(s)
    cos, sin = _cos_sin(s)
    dq, dwq = _norm_rope_grad(s["gq"], q, s["wq"], cos, sin, c)
    dk, dwk = _norm_rope_grad(s["gk"], k, s["wk"], cos, sin, c)
    return {"dq": dq.to(q.dtype), "dk": dk.to(k.dtype), "dwq": dwq, "dwk": dwk}


def _plain_attention(s):
    c = s["c"]
    B, Hq, Hk, D = c["B"], c["Hq"], c["Hk"], c["D"]
    at = s["table"].clamp(min=0).long()
    k = s["kc"].view(torch.uint8 if c["cache"] == "e4m3" else s["kc"].dtype)[at].view(s["kc"].dtype)
    v = s["vc"].view(torch.uint8 if c["cache"] == "e4m3" else s["vc"].dtype)[at].view(s["vc"].dtype)
    k = (k.reshape(B, -1, Hk, D).float() * s["ks"]).permute(0, 2, 3, 1).contiguous()
    v = (v.reshape(B, -1, Hk, D).float() * s["vs"]).permute(0, 2, 1, 3).contiguous()
    p = (s["q"].float() * D ** -0.5).view(B, Hk, Hq // Hk, D) @ k
    j = torch.arange(p.shape[-1], device=DEV)[None, :]
    n = s["lengths"].long()[:, None]
    seen = j < n
    if c["window"]:
        seen = seen & (j >= n - c["window"])
    p = p.masked_fill(~seen[:, None, None, :], -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = (p - m).exp()
    z = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(z == 0, torch.ones_like(z), z)
    return {"out": o.reshape(B, Hq, D).to(s["q"].dtype), "lse": (m + z.log()).reshape(B, Hq)}


def run(state):
    if own:
        return _own(state)
    op = state["c"]["op"]
    return {"lora": _plain_lora, "rope": _plain_rope, "rope_bwd": _plain_rope_bwd,
            "attention": _plain_attention}[op](state)


def work(case):
    c = case
    if c["op"] == "lora":
        M, N, K, R = c["M"], c["N"], c["K"], c["R"]
        used = min(c["L"], M if c["mix"] == "rows" else max(1, min(M, c["L"]) // 2))
        ob = 4 if c["out"] == "f32" else 2
        return {"bytes": 2 * (M * K + N * K + used * R * (K + N)) + ob * M * N,
                "flops": 2 * M * N * K + 2 * M * R * (K + N)}
    if c["op"] in ("rope", "rope_bwd"):
        T, Hq, Hk, D = c["T"], c["Hq"], c["Hk"], c["D"]
        if c["op"] == "rope":
            e = 1 if c["cache"] == "e4m3" else 2
            return {"bytes": T * D * (4 * Hq + 2 * Hk * (2 + e)), "flops": 10 * T * (Hq + Hk) * D}
        return {"bytes": 6 * T * D * (Hq + Hk), "flops": 20 * T * (Hq + Hk) * D}
    # lengths are even over 1 .. most: one is `most`, with more than two one is none
    B, most, w = c["B"], c["most"], c["window"]
    mean = (most + 1) / 2 if not w or w >= most else (w * (w + 1) / 2 + (most - w) * w) / most
    keys = (min(w, most) if w else most) + max(0, B - (2 if B > 2 else 1)) * mean
    e = 1 if c["cache"] == "e4m3" else 2
    return {"bytes": int(keys * c["Hk"] * c["D"] * 2 * e + 4 * B * c["Hq"] * c["D"]),
            "flops": int(4 * keys * c["Hq"] * c["D"])}


# ---- the definitions in 64 bits -------------------------------------------------------------------------

def _rotated(x, angle, layout, sign):
    """x (T, H, D) in 64 bits with pair j turned by sign * angle[:, j]: one rotation of the complex plane."""
    half = angle.shape[1]
    i = torch.arange(half, device=x.device)
    lo, hi = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
    z = torch.complex(x[..., lo], x[..., hi]) * torch.polar(torch.ones_like(angle), sign * angle)[:, None, :]
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    f64 = torch.float64
    if c["op"] == "lora":
        x = s["x"].to(f64)
        out = x @ s["w"].to(f64).T
        for a in range(c["L"]):
            at = torch.nonzero(s["rows"] == a)[:, 0]
            if at.numel():
                out[at] += float(s["scales"][a]) * ((x[at] @ s["a"][a].to(f64).T) @ s["b"][a].to(f64).T)
        return {"out": out}
    if c["op"] in ("rope", "rope_bwd"):
        T, Hq, Hk = c["T"], c["Hq"], c["Hk"]
        x = s["qkv"].to(f64).view(T, Hq + 2 * Hk, c["D"])
        angle = torch.outer(s["pos"].to(f64), s["inv_freq"])
        unit = lambda h: h / torch.sqrt(torch.square(h).mean(2, keepdim=True) + EPS)  # noqa: E731
        q, k, v = x.split([Hq, Hk, Hk], 1)
        if c["op"] == "rope":
            k = _rotated(unit(k) * s["wk"].to(f64), angle, c["layout"], 1.0)
            kc, vc = s["kc"].to(f64).flatten(0, 1), s["vc"].to(f64).flatten(0, 1)
            e4m3 = c["cache"] == "e4m3"
            for cache, new, scale in ((kc, k, K_SCALE), (vc, v, V_SCALE)):
                t = torch.nonzero(s["slots"] >= 0)[:, 0]
                cache[s["slots"][t].long()] = torch.clamp(new[t] / scale, -448.0, 448.0) if e4m3 else new[t]
            return {"q": _rotated(unit(q) * s["wq"].to(f64), angle, c["layout"], 1.0),
                    "k_cache": kc.view(s["kc"].shape), "v_cache": vc.view(s["vc"].shape)}
        got = {}
        for name, h, dy, w in (("q", q, s["gq"], s["wq"]), ("k", k, s["gk"], s["wk"])):
            dn = _rotated(dy.to(f64), angle, c["layout"], -1.0)
            norm = torch.sqrt(torch.square(h).mean(2, keepdim=True) + EPS)
            g = dn * w.to(f64)
            got["d" + name] = g / norm - h * (g * h).mean(2, keepdim=True) / norm ** 3
            got["dw" + name] = torch.einsum("thd,thd->d", dn, h / norm)
        return got
    B, Hq, Hk, D = c["B"], c["Hq"], c["Hk"], c["D"]
    out = torch.zeros((B, Hq, D), dtype=f64, device=DEV)
    lse = torch.full((B, Hq), -math.inf, dtype=f64, device=DEV)
    for b, n in enumerate(s["lengths"].tolist()):
        j = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device=DEV)
        if not j.numel():
            continue
        page, at = s["table"][b].long()[j // c["page"]], j % c["page"]
        for h in range(Hk):
            heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            k = s["kc"][:, :, h].view(torch.uint8 if c["cache"] == "e4m3" else s["kc"].dtype)[page, at]
            v = s["vc"][:, :, h].view(torch.uint8 if c["cache"] == "e4m3" else s["vc"].dtype)[page, at]
            k, v = k.view(s["kc"].dtype).to(f64) * s["ks"], v.view(s["vc"].dtype).to(f64) * s["vs"]
            score = (k @ s["q"][b, heads].to(f64).T) / math.sqrt(D)
            lse[b, heads] = torch.logsumexp(score, 0)
            out[b, heads] = torch.softmax(score, 0).T @ v
    return {"out": out, "lse": lse}
