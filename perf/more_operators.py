"""Cases of the operators of a server's step that drafts several tokens at once: the pages and slots of the
new tokens, the residual sum and norm before a product (in 16 bits, in 8 bits with block scales, and
backwards), the products of few rows with 4-bit weights, and the attention of a tree of drafted tokens over a
paged cache.

`run` computes them in their plain form (elementary torch operations in 32 bits, rounded once) or, with
`own`, through the library's entry points.  `exact` computes them from their definitions in 64 bits.

    norm       s = x + r;  y = w s / sqrt(mean(s^2) + eps) in 16 or 32 bits, s rounded and kept
    norm_mx    the same with y in E4M3 and one power of two for 32 elements, the smallest that takes them to
               at most 448
    norm_bwd   dx = (g - h mean(g h)) / sqrt(mean(s^2) + eps) + ds,  g = w dy,  h = s / sqrt(mean(s^2) + eps);
               dw = sum dy h
    w4         Out = X W^T, W = scale (q - zero) of 4-bit q in groups of K, or E2M1 elements times a power of
               two for 32
    tree       o = softmax(scale q k^T) v: the drafted tokens of a sequence are its last keys; each sees what
               came before them and the drafted tokens that its row of bits marks (a chain: itself and those
               before)
    plan       the sequences grow or shrink by `change`: pages from and to a stack of free ones, slots and
               positions of the new tokens
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
        # one token between two products: latency
        dict(name="norm_t1", op="norm", T=1, D=4096, dtype="bf16", out="bf16", weight="bf16", residual=True),
        # a long prompt before an 8-bit product: bound by memory
        dict(name="norm_mx_t8191", op="norm_mx", T=8191, D=4096, dtype="bf16", weight="bf16", residual=True),
        # training, a whole batch of tokens
        dict(name="norm_bwd_t8192", op="norm_bwd", T=8192, D=4096, dtype="bf16", weight="f32", residual=True),
        # one token of one request through a square projection: latency
        dict(name="w4_m1", op="w4", M=1, N=4096, K=4096, elem="u4", group=128, zeros=True, dtype="bf16", out="bf16"),
        # the drafted tokens of one request through a wide projection whose weights an 8-bit prompt also uses
        dict(name="w4_m12_e2m1", op="w4", M=12, N=12288, K=4096, elem="e2m1", group=32, zeros=False, dtype="bf16",
             out="bf16"),
        # a decode batch, logits of an odd vocabulary
        dict(name="w4_m48", op="w4", M=48, N=32003, K=4096, elem="u4", group=64, zeros=False, dtype="f16", out="f32"),
        # one request, a small tree of drafts on a short context: latency
        dict(name="tree_b1", op="tree", B=1, Hq=32, Hk=8, D=128, most=700, nodes=9, page=16, dtype="bf16",
             cache="same", window=0, kind="tree"),
        # a batch of requests with trees of up to 64 drafts
        dict(name="tree_b16", op="tree", B=16, Hq=32, Hk=8, D=128, most=4096, nodes=64, page=16, dtype="bf16",
             cache="same", window=0, kind="tree"),
        # few drafts in a row on a long context: split over its length
        dict(name="chain_b2_long", op="tree", B=2, Hq=32, Hk=8, D=128, most=65537, nodes=5, page=64, dtype="f16",
             cache="same", window=0, kind="chain"),
        # a decode batch over an 8-bit cache
        dict(name="tree_b32_e4m3", op="tree", B=32, Hq=64, Hk=8, D=128, most=4096, nodes=16, page=64, dtype="bf16",
             cache="e4m3", window=0, kind="tree"),
        # a step's drafts of every request get their places, and none is kept
        dict(name="plan_drafts", op="plan", B=64, most=4096, page=16, grow=8, finish=0),
        # prompts are admitted while other requests end
        dict(name="plan_prompts", op="plan", B=256, most=8192, page=16, grow=2000, finish=64),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_mx", "norm_bwd", "w4", "w4", "tree", "tree", "plan"])
    dtype = rng.choice(["bf16", "f16"])
    if op.startswith("norm"):
        D = 32 * _log(rng, 2, 256) if op == "norm_mx" else 8 * _log(rng, 8, 1024)
        c = dict(op=op, T=_log(rng, 1, min(8192, (1 << 25) // D)), D=D, dtype=dtype, weight=rng.choice([dtype, "f32"]),
                 residual=rng.random() < 0.75)
        if op == "norm":
            c.update(out=rng.choice([dtype, dtype, "f32"]))
        return c
    if op == "w4":
        elem = rng.choice(["u4", "u4", "e2m1"])
        group = 32 if elem == "e2m1" else rng.choice([32, 64, 128])
        M, K = _log(rng, 1, 64), group * (_log(rng, 512, 8192) // group)
        N = _log(rng, 64, min(16384, 131_000_000 // K, 6_290_000_000 // (K * M)))
        return dict(op=op, M=M, N=N, K=K, elem=elem, group=group,
                    zeros=elem == "u4" and rng.random() < 0.5, dtype=dtype, out=rng.choice([dtype, "f32"]))
    if op == "tree":
        B, Hk, nodes = _log(rng, 1, 32), rng.choice([1, 2, 4, 8]), _log(rng, 1, 64)
        Hq = Hk * rng.choice([1, 2, 4, 8])
        most = _log(rng, nodes, min(65537, (1 << 26) // (B * Hq * nodes), (1 << 20) // (B * Hk)))
        return dict(op=op, B=B, Hq=Hq, Hk=Hk, D=rng.choice([64, 80, 96, 128, 128]), most=most, nodes=nodes,
                    page=rng.choice([8, 16, 64, 128]), dtype=dtype, cache=rng.choice(["same", "e4m3"]),
                    window=rng.choice([0, 0, max(1, most // 3)]), kind=rng.choice(["tree", "tree", "chain"]))
    B = _log(rng, 1, 256)
    page = rng.choice([1, 8, 16, 24, 64])
    return dict(op=op, B=B, most=_log(rng, 64, min(8192, 512 * page)), page=page, grow=_log(rng, 1, min(2000, 128 * page)),
                finish=rng.choice([0, B // 4]))


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, sigma, dt):
    return (torch.randn(shape, generator=g, device=DEV) * sigma).to(dt)


def _cache(shape, g, kind, dt):
    """Keys or values already in a cache; 8-bit ones as bytes."""
    if kind == "e4m3":
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16) * 16.0
        return x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float16).to(dt)


def _prepare_norm(c, g):
    T, D, dt = c["T"], c["D"], DT[c["dtype"]]
    s = dict(x=_normal((T, D), g, 1.0, dt), r=_normal((T, D), g, 4.0, dt) if c["residual"] else None,
             w=(1 + 0.2 * torch.randn((D,), generator=g, device=DEV)).to(DT[c["weight"]]),
             sum=torch.empty((T, D), dtype=dt, device=DEV))
    if c["op"] == "norm":
        s["y"] = torch.empty((T, D), dtype=DT[c["out"]], device=DEV)
    elif c["op"] == "norm_mx":
        s["y"] = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=DEV)
        s["scale"] = torch.empty((T, D // 32), dtype=torch.float8_e8m0fnu, device=DEV)
    else:
        s["dy"] = _normal((T, D), g, 1.0, dt)
        s["dx"] = torch.empty((T, D), dtype=dt, device=DEV)
        s["dw"] = torch.empty((D,), dtype=torch.float32, device=DEV)
    return s


def _prepare_w4(c, g):
    M, N, K, G, dt = c["M"], c["N"], c["K"], c["group"], DT[c["dtype"]]
    s = dict(x=_normal((M, K), g, 1.0, dt),
             w=torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8), zeros=None,
             out=torch.empty((M, N), dtype=DT[c["out"]], device=DEV))
    if c["elem"] == "e2m1":  # powers of two around 2^-8
        s["scales"] = torch.randint(117, 122, (N, K // G), generator=g, device=DEV, dtype=torch.uint8)
    else:
        s["scales"] = ((0.5 + torch.rand((N, K // G), generator=g, device=DEV)) * (0.2 * K ** -0.5)).to(dt)
        if c["zeros"]:
            s["zeros"] = torch.randint(4, 12, (N, K // G), generator=g, device=DEV, dtype=torch.uint8)
    return s


def _prepare_tree(c, g):
    B, Hq, Hk, D, most, page, n = c["B"], c["Hq"], c["Hk"], c["D"], c["most"], c["page"], c["nodes"]
    dt = DT[c["dtype"]]
    per = -(-most // page)
    pages = B * per
    s = dict(q=_normal((B * n, Hq, D), g, 1.0, dt), kc=_cache((pages, page, Hk, D), g, c["cache"], dt),
             vc=_cache((pages, page, Hk, D), g, c["cache"], dt))
    # drafted tokens of every sequence: up to n, of one sequence n, of another (where there are three) none
    count = torch.randint(1, n + 1, (B,), generator=g, device=DEV)
    count[0] = n
    if B > 2:
        count[1] = 0
    s["starts"] = torch.cat((torch.zeros_like(count[:1]), count.cumsum(0))).to(torch.int32)
    lengths = count + (torch.rand((B,), generator=g, device=DEV) * (most - count + 1)).long()
    lengths[0] = most
    s["lengths"] = lengths.to(torch.int32)
    table = torch.randperm(pages, generator=g, device=DEV).view(B, per)
    used = torch.arange(per, device=DEV)[None, :] * page < lengths[:, None]
    s["table"] = torch.where(used, table, -1).to(torch.int32).contiguous()
    s["tree"] = None
    if c["kind"] == "tree":  # every node hangs on an earlier one, or on the context
        up = (torch.rand((B, n), generator=g, device=DEV) * torch.arange(1, n + 1, device=DEV)).long() - 1
        own_bit = torch.bitwise_left_shift(torch.ones((), dtype=torch.int64, device=DEV), torch.arange(n, device=DEV))
        seen = torch.zeros((B, n), dtype=torch.int64, device=DEV)
        for i in range(n):
            seen[:, i] = own_bit[i] | torch.where(up[:, i] < 0, 0, seen.gather(1, up[:, i:i + 1].clamp(min=0))[:, 0])
        b, i = _rows(s["starts"], B * n)
        s["tree"] = seen[b, i.clamp(max=n - 1)][:, None].contiguous()
    s["out"] = torch.zeros((B * n, Hq, D), dtype=dt, device=DEV)
    s["lse"] = torch.zeros((B * n, Hq), dtype=torch.float32, device=DEV)
    s["ks"], s["vs"] = (K_SCALE, V_SCALE) if c["cache"] == "e4m3" else (1.0, 1.0)
    return s


def _prepare_plan(c, g):
    B, most, page, grow, finish = c["B"], c["most"], c["page"], c["grow"], c["finish"]
    per = -(-(most + grow) // page)
    lengths = torch.randint(0, most + 1, (B,), generator=g, device=DEV)
    change = torch.randint(0, grow + 1, (B,), generator=g, device=DEV)
    change[0] = grow
    ends = torch.randperm(B, generator=g, device=DEV)[:finish]
    change[ends] = -lengths[ends]
    used = torch.arange(per, device=DEV)[None, :] * page < lengths[:, None]
    order = torch.randperm(B * per, generator=g, device=DEV)
    taken = used.flatten()
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    # pages that no sequence holds, in any order, at the bottom of a stack with room for all
    free = torch.cat((order[~taken], torch.full((int(taken.sum()),), -1, device=DEV)))
    T = B * grow
    return dict(lengths=i32(lengths), change=i32(change), back=i32(-change), table=i32(torch.where(used, order.view(B, per), -1)),
                free=i32(free), count=i32((~taken).sum().view(1)), T=T,
                starts=torch.empty((2, B + 1), dtype=torch.int32, device=DEV),
                slots=torch.empty((2, T), dtype=torch.int32, device=DEV),
                positions=torch.empty((2, T), dtype=torch.int32, device=DEV))


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    kind = "norm" if c["op"].startswith("norm") else c["op"]
    s = {"norm": _prepare_norm, "w4": _prepare_w4, "tree": _prepare_tree, "plan": _prepare_plan}[kind](c, g)
    s["c"] = c
    return s


# ---- the library's entry points -------------------------------------------------------------------------

def _own(s):
    import tensor_core_matrix_amd as tcm
    c = s["c"]
    op = c["op"]
    if op == "norm":
        tcm.add_rms_norm(s["x"], s["w"], residual=s["r"], eps=EPS, out=s["y"], sum_out=s["sum"])
        return {"y": s["y"], "sum": s["sum"]}
    if op == "norm_mx":
        tcm.add_rms_norm_mx_fp8(s["x"], s["w"], residual=s["r"], eps=EPS, out=s["y"], scale=s["scale"],
                                sum_out=s["sum"])
        return {"y": s["y"], "scale": s["scale"], "sum": s["sum"]}
    if op == "norm_bwd":
        tcm.add_rms_norm_bwd(s["dy"], s["x"], s["w"], dsum=s["r"], eps=EPS, dx=s["dx"], dw=s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "w4":
        tcm.gemm_w4(s["x"], s["w"], s["scales"], s["zeros"], elem=c["elem"], out=s["out"])
        return {"out": s["out"]}
    if op == "tree":
        tcm.paged_tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["lengths"], s["starts"], c["nodes"],
                                 tree=s["tree"], window=c["window"], max_len=c["most"], k_scale=s["ks"],
                                 v_scale=s["vs"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    # the change and its undoing: afterwards lengths, table and stack are as they were
    one = lambda change, i: tcm.cache_plan(s["lengths"], change, s["table"], s["free"], s["count"], c["page"],  # noqa: E731
                                           starts=s["starts"][i], slots=s["slots"][i], positions=s["positions"][i])
    one(s["change"], 0)
    one(s["back"], 1)
    return {k: s[k] for k in ("starts", "slots", "positions", "lengths", "table", "free", "count")}


# ---- the plain forms ------------------------------------------------------------------------------------

def _sum(s):
    return s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()


def _normed(s):
    t = _sum(s)
    return t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS) * s["w"].float(), t


def _plain_norm(s):
    y, t = _normed(s)
    return {"y": y.to(s["y"].dtype), "sum": t.to(s["x"].dtype)}


def _plain_norm_mx(s):
    y, t = _normed(s)
    y = y.view(y.shape[0], -1, 32)
    m, e = torch.frexp(y.abs().amax(-1))
    # 448 = 0.875 * 2^9; a block of zeros has the least scale
    e = torch.where(m == 0, -127, (e - 9 + (m > 0.875)).clamp(-127, 127))
    q = torch.ldexp(y, -e[..., None]).to(torch.float8_e4m3fn)
    return {"y": q.view(s["y"].shape), "scale": (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu),
            "sum": t.to(s["x"].dtype)}


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    h, g = x * r, dy * s["w"].float()
    dx = r * (g - h * (g * h).mean(-1, keepdim=True))
    if s["r"] is not None:
        dx = dx + s["r"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * h).sum(0)}


def _weights(s):
    c = s["c"]
    q = torch.stack((s["w"] & 15, s["w"] >> 4), -1).view(c["N"], -1, c["group"])
    if c["elem"] == "e2m1":
        value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
        return (value[q.int()] * torch.exp2(s["scales"].float() - 127)[..., None]).view(c["N"], c["K"])
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    return ((q.float() - zero) * s["scales"].float()[..., None]).view(c["N"], c["K"])


def _plain_w4(s):
    return {"out": (s["x"].float() @ _weights(s).t()).to(s["out"].dtype)}


def _rows(starts, T):
    """The sequence of every row and its number there (rows behind the last sequence: of the last)."""
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(starts[1:], t.to(torch.int32), right=True).clamp(max=starts.numel() - 2)
    return b, t - starts[b]


def _plain_tree(s):
    c = s["c"]
    B, Hq, Hk, D, n = c["B"], c["Hq"], c["Hk"], c["D"], c["nodes"]
    at = s["table"].clamp(min=0).long()
    raw = torch.uint8 if c["cache"] == "e4m3" else s["kc"].dtype
    k = s["kc"].view(raw)[at].view(s["kc"].dtype).reshape(B, -1, Hk, D).float() * s["ks"]
    v = s["vc"].view(raw)[at].view(s["vc"].dtype).reshape(B, -1, Hk, D).float() * s["vs"]
    k, v = k.permute(0, 2, 3, 1).contiguous(), v.permute(0, 2, 1, 3).contiguous()
    # every sequence's rows, padded to n
    starts, lengths = s["starts"].long(), s["lengths"].long()
    count = starts[1:] - starts[:-1]
    i = torch.arange(n, device=DEV)
    row = (starts[:-1, None] + i).clamp(max=B * n - 1)
    q = s["q"][row].float() * D ** -0.5
    p = q.view(B, n, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D).contiguous() @ k
    p = p.view(B, Hk, Hq // Hk, n, -1)
    # which keys a row sees: of the context, and of the drafted tokens by number j - context
    j = torch.arange(p.shape[-1], device=DEV)
    context = (lengths - count)[:, None, None]
    node = j - context
    if s["tree"] is None:
        seen = node <= i[:, None]
        place = context + i[:, None]
        if c["window"]:
            seen = seen & (j > place - c["window"])
    else:
        bits = s["tree"][:, 0][row]
        marked = (torch.bitwise_right_shift(bits[:, :, None], node.clamp(0, 63)) & 1) == 1
        old = node < 0
        if c["window"]:
            depth = ((bits[:, :, None] >> i) & 1 & (i < count[:, None, None])).sum(-1, keepdim=True)
            old = old & (j > context + depth - 1 - c["window"])
        seen = old | ((node >= 0) & marked)
    seen = seen & (j < lengths[:, None, None])
    p = p.masked_fill(~seen[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = (p - m).exp()
    z = p.sum(-1, keepdim=True)
    o = (p.view(B, Hk, -1, p.shape[-1]) @ v).view(B, Hk, Hq // Hk, n, D) / torch.where(z == 0, torch.ones_like(z), z)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    lse = (m + z.log()).permute(0, 3, 1, 2, 4).reshape(B, n, Hq)
    b, i = _rows(s["starts"], B * n)
    live = torch.arange(B * n, device=DEV) < starts[-1]
    i = i.clamp(max=n - 1)
    return {"out": torch.where(live[:, None, None], o[b, i].to(s["q"].dtype), s["out"]),
            "lse": torch.where(live[:, None], lse[b, i], s["lse"])}


def _step(lengths, change, table, free, count, page, T):
    """One change of the lengths: new lengths, table, stack and its count, and the new tokens' starts, slots
    and positions."""
    B, per = table.shape
    end = (lengths + change).clamp(0, per * page)
    first, last = (lengths + page - 1) // page, (end + page - 1) // page
    i = torch.arange(per, device=DEV)
    drop = (i >= last[:, None]) & (i < first[:, None]) & (table >= 0)
    order = drop.flatten().cumsum(0)
    top = count + order[-1]
    # (what is not dropped goes to a place behind the stack)
    to = torch.where(drop.flatten(), top - order, free.numel())
    free = torch.cat((free, free[:1])).scatter(0, to, table.flatten())[:-1]
    table = torch.where((i >= last[:, None]) & (i < first[:, None]), -1, table)
    need = (i >= first[:, None]) & (i < last[:, None])
    order = need.flatten().cumsum(0)
    page_at = (top - order).view(B, per)
    table = torch.where(need, torch.where(page_at >= 0, free[page_at.clamp(0, free.numel() - 1)], -1), table)
    new = (end - lengths).clamp(min=0)
    starts = torch.cat((torch.zeros_like(new[:1]), new.cumsum(0)))
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(starts[1:], t, right=True).clamp(max=B - 1)
    place = lengths[b] + t - starts[b]
    live = t < starts[-1]
    at = table[b, torch.where(live, place // page, 0)]
    slots = torch.where(live & (at >= 0), at * page + place % page, -1)
    return end, table, free, (top - order[-1]).clamp(min=0), starts, slots, torch.where(live, place, 0)


def _plain_plan(s):
    page, T = s["c"]["page"], s["T"]
    lengths, table, free, count, st0, sl0, po0 = _step(s["lengths"].long(), s["change"].long(), s["table"].long(),
                                                       s["free"].long(), s["count"].long(), page, T)
    lengths, table, free, count, st1, sl1, po1 = _step(lengths, s["back"].long(), table, free, count, page, T)
    i32 = lambda *t: torch.stack(t).to(torch.int32)  # noqa: E731
    return {"starts": i32(st0, st1), "slots": i32(sl0, sl1), "positions": i32(po0, po1),
            "lengths": lengths.to(torch.int32), "table": table.to(torch.int32), "free": free.to(torch.int32),
            "count": count.to(torch.int32)}


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_mx": _plain_norm_mx, "norm_bwd": _plain_norm_bwd, "w4": _plain_w4,
            "tree": _plain_tree, "plan": _plain_plan}[state["c"]["op"]](state)


def work(case):
    c = case
    if c["op"].startswith("norm"):
        T, D, r = c["T"], c["D"], int(c["residual"])
        # x, the residual (its gradient), the sum; backwards dy, x, ds and dx
        each = {"norm": 4 + 2 * r + (4 if c.get("out") == "f32" else 2), "norm_mx": 4 + 2 * r + 1 + 1 / 32,
                "norm_bwd": 6 + 2 * r}[c["op"]]
        return {"bytes": int(T * D * each + D * (4 if c["weight"] == "f32" else 2)), "flops": 10 * T * D}
    if c["op"] == "w4":
        M, N, K, G = c["M"], c["N"], c["K"], c["group"]
        scale = 1 if c["elem"] == "e2m1" else 3 if c["zeros"] else 2
        return {"bytes": N * K // 2 + N * (K // G) * scale + 2 * M * K + (4 if c["out"] == "f32" else 2) * M * N,
                "flops": 2 * M * N * K}
    if c["op"] == "tree":
        # drafts are even over 1 .. nodes and lengths over what holds them: one sequence has the most of both,
        # with more than two one has no drafts, and none of its keys is read
        B, most, n = c["B"], c["most"], c["nodes"]
        rest = max(0, B - (2 if B > 2 else 1))
        w = c["window"] or most
        mean = min((n + 1) / 2 + (most - n) / 2, w)
        keys, e = min(most, w) + rest * mean, 1 if c["cache"] == "e4m3" else 2
        rows = n + rest * (n + 1) / 2
        return {"bytes": int(keys * c["Hk"] * c["D"] * 2 * e + 4 * rows * c["Hq"] * c["D"]),
                "flops": int(4 * (n * min(most, w) + rest * (n + 1) / 2 * mean) * c["Hq"] * c["D"])}
    # both directions: lengths and changes, pages and new tokens' slots and positions, even over 0 .. grow
    tokens = c["B"] * c["grow"]
    return {"bytes": int(2 * (20 * c["B"] + 8 * tokens + 12 * (tokens // (2 * c["page"]) + c["B"]))), "flops": 4 * tokens}


# ---- the definitions in 64 bits -------------------------------------------------------------------------

def _exact_norm(c, s):
    f64 = torch.float64
    x, w = s["x"].to(f64), s["w"].to(f64)
    if c["op"] == "norm_bwd":
        norm = torch.sqrt(torch.square(x).mean(1, keepdim=True) + EPS)
        dy = s["dy"].to(f64)
        dot = torch.einsum("td,d,td->t", dy, w, x)[:, None] / c["D"]
        dx = dy * w / norm - x * dot / norm ** 3
        return {"dx": dx if s["r"] is None else dx + s["r"].to(f64), "dw": torch.sum(dy * (x / norm), 0)}
    if s["r"] is not None:
        x = x + s["r"].to(f64)
    y = w * (x / torch.sqrt(torch.square(x).mean(1, keepdim=True) + EPS))
    if c["op"] == "norm":
        return {"y": y, "sum": x}
    top = y.view(c["T"], -1, 32).abs().amax(2)
    scale = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(-127.0, 127.0))
    return {"y": y / scale.repeat_interleave(32, 1), "scale": scale, "sum": x}


def _exact_w4(c, s):
    f64 = torch.float64
    q = torch.empty((c["N"], c["K"]), dtype=f64, device=DEV)
    q[:, 0::2], q[:, 1::2] = s["w"] % 16, s["w"] // 16
    if c["elem"] == "e2m1":  # sign, two bits of exponent, one of mantissa
        sign, m = 1 - 2 * torch.floor(q / 8), q % 8
        e = torch.floor(m / 2)
        q = sign * torch.where(e == 0, m % 2 * 0.5, (1 + m % 2 * 0.5) * torch.exp2(e - 1))
        scale = torch.exp2(s["scales"].to(f64) - 127)
    else:
        q -= 8 if s["zeros"] is None else s["zeros"].to(f64).repeat_interleave(c["group"], 1)
        scale = s["scales"].to(f64)
    return {"out": s["x"].to(f64) @ (q * scale.repeat_interleave(c["group"], 1)).T}


def _exact_tree(c, s):
    f64 = torch.float64
    Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
    out, lse = s["out"].to(f64), s["lse"].to(f64)
    starts = s["starts"].tolist()
    raw = torch.uint8 if c["cache"] == "e4m3" else s["kc"].dtype
    for b, length in enumerate(s["lengths"].tolist()):
        n = starts[b + 1] - starts[b]
        if n == 0:
            continue
        j = torch.arange(length, device=DEV)
        sees = torch.ones((n, length), dtype=torch.bool, device=DEV)
        if s["tree"] is None:
            sees[:, length - n:] = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()
            depth = torch.arange(1, n + 1, device=DEV)
        else:
            bits = s["tree"][starts[b]:starts[b + 1], 0].tolist()
            mine = torch.tensor([[(m >> i) & 1 for i in range(n)] for m in bits], dtype=torch.bool, device=DEV)
            sees[:, length - n:] = mine
            depth = mine.sum(1)
        if c["window"]:
            far = j <= (length - n + depth - 1 - c["window"])[:, None]
            if s["tree"] is not None:
                far[:, length - n:] = False
            sees &= ~far
        page, at = s["table"][b].long()[j // c["page"]], j % c["page"]
        for h in range(Hk):
            heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            k = s["kc"][:, :, h].view(raw)[page, at].view(s["kc"].dtype).to(f64) * s["ks"]
            v = s["vc"][:, :, h].view(raw)[page, at].view(s["vc"].dtype).to(f64) * s["vs"]
            q = s["q"][starts[b]:starts[b + 1], heads].to(f64).flatten(0, 1)
            score = (q @ k.T / math.sqrt(D)).masked_fill(~sees.repeat_interleave(Hq // Hk, 0), -math.inf)
            lse[starts[b]:starts[b + 1], heads] = torch.logsumexp(score, 1).view(n, -1)
            out[starts[b]:starts[b + 1], heads] = (torch.softmax(score, 1).nan_to_num() @ v).view(n, -1, D)
    return {"out": out, "lse": lse}


def exact(case, seed):
    c = dict(case)
    if c["op"] == "plan":  # whole numbers
        return None
    s = prepare(c, seed)
    return (_exact_norm if c["op"].startswith("norm") else _exact_w4 if c["op"] == "w4" else _exact_tree)(c, s)
