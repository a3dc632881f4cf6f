"""Measured cases of the draft-attention operators.

Each case is one call of one operator as a draft step makes it: the cos|sin
table (``table``), rotary positions with the K/V insert (``rope``), the
drafted tokens' attention over the paged cache (``attention``), the attention
weight each cached token received (``weight``) and the eviction by that weight
(``evict``).  ``own`` false computes the plain form in elementary torch
operations; true makes the framework's calls.
"""

import math

import torch

own = False

FP8_MAX = 448.0


# ------------------------------------------------------------------ cases


def listed():
    return [
        # the table of a 131,072-position drafter, frequencies scaled by parts
        dict(name="table_131072", op="table", positions=131072, first=0, rotary=64, theta=1e6, kind="by_parts", factor=4.0, fp32=False),
        # a window of far positions in fp32, a whole 128-dim head rotated
        dict(name="table_far_fp32", op="table", positions=4096, first=1 << 20, rotary=128, theta=1e4, kind="bands", factor=8.0, fp32=True),
        # one request's seven drafted tokens, half layout, inserted (latency)
        dict(name="rope_draft_one", op="rope", tokens=7, heads=64, kv_heads=8, dim=128, rotary=64, layout="half", block=16, fp8=False, insert=True, inverse=False),
        # a prefill batch, interleaved pairs, into an fp8 cache
        dict(name="rope_prefill_fp8", op="rope", tokens=8192, heads=32, kv_heads=8, dim=128, rotary=32, layout="interleaved", block=64, fp8=True, insert=True, inverse=False),
        # one request's seven drafted tokens over a short context (latency)
        dict(name="attn_one", op="attention", requests=1, q_min=7, q_max=7, heads=64, kv_heads=8, dim=128, ctx_min=300, ctx_max=300, block=16, fp8=False, mask="dense"),
        # a draft step of 64 requests, seven drafted tokens each
        dict(name="attn_draft_step", op="attention", requests=64, q_min=7, q_max=7, heads=64, kv_heads=8, dim=128, ctx_min=1024, ctx_max=8192, block=16, fp8=False, mask="dense"),
        # ragged trees over an fp8 cache, requests without a context among them
        dict(name="attn_trees_fp8", op="attention", requests=17, q_min=1, q_max=63, heads=40, kv_heads=8, dim=128, ctx_min=0, ctx_max=16384, block=64, fp8=True, mask="tree"),
        # trees of 64 over two long contexts
        dict(name="attn_long", op="attention", requests=2, q_min=64, q_max=64, heads=32, kv_heads=4, dim=128, ctx_min=100003, ctx_max=131072, block=128, fp8=False, mask="tree"),
        # the weight a draft step's context tokens received
        dict(name="weight_draft_step", op="weight", requests=64, q_min=7, q_max=7, heads=64, kv_heads=8, dim=128, ctx_min=1024, ctx_max=8192, block=16, fp8=False, mask="dense"),
        # the same over two long fp8 contexts
        dict(name="weight_long_fp8", op="weight", requests=2, q_min=5, q_max=9, heads=32, kv_heads=4, dim=128, ctx_min=65536, ctx_max=131072, block=128, fp8=True, mask="dense"),
        # a serving batch 256 tokens over its budget
        dict(name="evict_serving", op="evict", requests=64, kv_heads=8, dim=128, ctx_min=4100, ctx_max=4352, budget=4096, block=16, fp8=False),
        # two long contexts halved
        dict(name="evict_long", op="evict", requests=2, kv_heads=4, dim=128, ctx_min=131000, ctx_max=131072, budget=65536, block=128, fp8=False),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["table", "rope", "attention", "attention", "weight", "evict"])
    dim = rng.choice([64, 128, 128, 256])
    block = rng.choice([1, 3, 16, 16, 32, 48, 64, 100, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    fp8 = rng.random() < 0.5
    if op == "table":
        rotary = rng.choice([2, 6, 16, 32, 64, 100, 128, 256])
        return dict(op=op, positions=_log(rng, 1, 131072 * 32 // rotary), first=_log(rng, 1, 1 << 20) - 1, rotary=rotary,
                    theta=rng.choice([1e4, 5e5, 1e6]), kind=rng.choice(["none", "linear", "by_parts", "bands"]),
                    factor=rng.choice([2.0, 4.0, 8.0, 32.0]), fp32=rng.random() < 0.5)
    if op == "rope":
        heads = kv_heads * rng.choice([1, 3, 5, 8])
        most = max(1, (8192 * 48 * 128) // ((heads + 2 * kv_heads) * dim))
        return dict(op=op, tokens=_log(rng, 1, min(8192, most)), heads=heads, kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice([r for r in (2, 6, 16, 18, 32, 50, 64, 128, 256) if r <= dim]),
                    layout=rng.choice(["half", "interleaved"]), block=block, fp8=fp8, insert=rng.random() < 0.6,
                    inverse=rng.random() < 0.3)
    if op == "evict":
        requests = _log(rng, 1, 64)
        longest = max(64, min(131072, (1 << 28) // (requests * kv_heads * dim)))
        ctx = _log(rng, 40, longest)
        return dict(op=op, requests=requests, kv_heads=kv_heads, dim=dim, ctx_min=max(1, ctx // 2), ctx_max=ctx,
                    budget=rng.randint(24, ctx), block=block, fp8=fp8)
    requests = _log(rng, 1, 64)
    group = rng.choice([1, 2, 3, 5, 8, 16])
    q_max = _log(rng, 1, 64)
    rows = q_max * group * kv_heads
    longest = min(131072, (1 << 28) // (requests * kv_heads * dim), (1 << 29) // (requests * rows))
    ctx = _log(rng, 1, max(64, longest))
    return dict(op=op, requests=requests, q_min=rng.randint(1, q_max), q_max=q_max, heads=kv_heads * group, kv_heads=kv_heads,
                dim=dim, ctx_min=rng.choice([1, ctx // 2 + 1]), ctx_max=ctx, block=block, fp8=fp8,
                mask=rng.choice(["dense", "causal", "tree"]) if op == "attention" else "dense")


def _spread(n, lo, hi, step):
    """n whole numbers over [lo, hi], over their logarithm: the same ones each time, the first the largest."""
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [hi if i == 0 else min(hi, max(lo, int(round(math.exp(b - (b - a) * ((i * step) % 1.0)) - 1)))) for i in range(n)]


def _lengths(c):
    ctx = _spread(c["requests"], c["ctx_min"], c["ctx_max"], 0.618034)
    if c["ctx_min"] == 0 and c["requests"] > 2:
        ctx[2] = 0
    q = _spread(c["requests"], c["q_min"], c["q_max"], 0.414214) if "q_min" in c else [0] * c["requests"]
    return ctx, q


def _scaling(c):
    """The scaling of a table case as the framework's call takes it."""
    return {"none": None,
            "linear": dict(kind="linear", factor=c["factor"]),
            "by_parts": dict(kind="by_parts", factor=c["factor"], original_positions=32768, beta_fast=32.0, beta_slow=1.0),
            "bands": dict(kind="bands", factor=c["factor"], original_positions=8192, low_freq_factor=1.0, high_freq_factor=4.0),
            }[c["kind"]]


# ------------------------------------------------------------------ inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cache(c, blocks, g):
    """A paged cache with every slot written, the blocks that no request holds among them."""
    shape = (blocks, c["kv_heads"], c["block"], 2 * c["dim"])
    k_scale = torch.rand(1, generator=g, device="cuda") * 0.04 + 0.01
    v_scale = torch.rand(1, generator=g, device="cuda") * 0.04 + 0.01
    if not c["fp8"]:
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16), k_scale, v_scale
    cache = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    D = c["dim"]
    for half, s in ((slice(0, D), k_scale), (slice(D, 2 * D), v_scale)):
        x = torch.randn(shape[:3] + (D,), generator=g, device="cuda", dtype=torch.bfloat16)
        cache[..., half] = (x / s.to(x.dtype)).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return cache.view(torch.uint8), k_scale, v_scale


def _block_table(c, need, g):
    """Every request's shuffled physical blocks."""
    per = max(1, max(-(-n // c["block"]) for n in need))
    count = sum(-(-n // c["block"]) for n in need)
    blocks = count + 3
    order = torch.randperm(blocks, generator=g, device="cuda")[:count].to(torch.int32).cpu()
    table = torch.full((len(need), per), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        m = -(-n // c["block"])
        table[b, :m] = order[at:at + m]
        at += m
    return table.cuda(), blocks


def _tree(q, words, seed):
    """Bit j of row i: node j is node i or one of its ancestors."""
    import random

    r = random.Random(seed)
    rows = []
    for n in q:
        seen = []
        for i in range(n):
            up = r.randrange(-1, i) if i else -1
            seen.append((seen[up] if up >= 0 else 0) | (1 << i))
        rows += seen
    out = torch.empty((len(rows), words), dtype=torch.int64)
    for t, m in enumerate(rows):
        for w in range(words):
            x = (m >> (64 * w)) & ((1 << 64) - 1)
            out[t, w] = x - (1 << 64) if x >= 1 << 63 else x
    return out.cuda()


def prepare(case, seed):
    c, g = case, _generator(seed)
    if c["op"] == "table":
        # the table's first position is what differs from one call to the next
        return dict(op="table", c=c, first=c["first"] + seed % 64)
    if c["op"] == "rope":
        T, Hq, Hk, D, r = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["rotary"]
        qkv = torch.randn((T, (Hq + 2 * Hk) * D), generator=g, device="cuda", dtype=torch.bfloat16) * 2
        rows = 32768
        angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * (1e6 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r))
        s = dict(op="rope", c=c, table=torch.cat([angle.cos(), angle.sin()], 1).to(torch.bfloat16),
                 positions=torch.randint(0, rows, (T,), generator=g, device="cuda"))
        s["q"], s["k"], s["v"] = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hk * D, Hk * D], 1))
        if c["insert"]:
            blocks = -(-T // c["block"]) + 5
            s["cache"] = torch.zeros((blocks, Hk, c["block"], 2 * D), device="cuda", dtype=torch.uint8 if c["fp8"] else torch.bfloat16)
            s["slots"] = torch.randperm(blocks * c["block"], generator=g, device="cuda")[:T].contiguous()
            if T > 1:
                s["slots"][T // 2::50] = -1  # padding
            s["k_scale"] = torch.rand(1, generator=g, device="cuda") * 0.45 + 0.05
            s["v_scale"] = torch.rand(1, generator=g, device="cuda") * 0.45 + 0.05
        return s
    ctx, q = _lengths(c)
    table, blocks = _block_table(c, [n + m for n, m in zip(ctx, q)], g)
    cache, k_scale, v_scale = _cache(c, blocks, g)
    s = dict(op=c["op"], c=c, cache=cache, k_scale=k_scale, v_scale=v_scale, table=table,
             ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"), longest=max(n + m for n, m in zip(ctx, q)))
    if c["op"] == "evict":
        B, H, S = c["requests"], c["kv_heads"], max(ctx)
        s["weights"] = torch.rand((B, H, S), generator=g, device="cuda") ** 4
        # what an earlier eviction left: tokens in no order, the newest last
        s["positions"] = torch.argsort(torch.rand((B, H, S), generator=g, device="cuda"), -1).to(torch.int32)
        s["seen"] = torch.full((B,), S, dtype=torch.int32, device="cuda")
        s["weights_out"], s["positions_out"] = torch.empty_like(s["weights"]), torch.empty_like(s["positions"])
        return s
    T = sum(q)
    start = [0]
    for m in q:
        start.append(start[-1] + m)
    s["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    s["q"] = torch.randn((T, c["heads"], c["dim"]), generator=g, device="cuda", dtype=torch.bfloat16) * 2
    s["mask"] = _tree(q, -(-c["q_max"] // 64), seed) if c["mask"] == "tree" else None
    # where each query sits, for the plain form
    s["of"] = torch.tensor([b for b, m in enumerate(q) for _ in range(m)], device="cuda")
    s["node"] = torch.tensor([i for m in q for i in range(m)], device="cuda")
    if c["op"] == "weight":
        s["lse"] = _plain_scores(s)[0].logsumexp(-1).to(torch.float32)
        s["weights"] = torch.rand((c["requests"], c["kv_heads"], max(ctx)), generator=g, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms


def _plain_frequencies(c, r):
    f = torch.tensor(c["theta"], dtype=torch.float64, device="cuda") ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
    s, amp = _scaling(c), 1.0
    if s is None:
        return f, amp
    if s["kind"] == "linear":
        return f / s["factor"], amp
    turns = s["original_positions"] * f / (2 * math.pi)  # turns over the original length
    if s["kind"] == "by_parts":
        # dims that turn over beta_fast times keep their frequency, those under beta_slow are stretched; a ramp over the dims between
        dim_of = lambda t: r * math.log(s["original_positions"] / (t * 2 * math.pi)) / (2 * math.log(c["theta"]))  # noqa: E731
        lo, hi = max(0, math.floor(dim_of(s["beta_fast"]))), min(r - 1, math.ceil(dim_of(s["beta_slow"])))
        ramp = ((torch.arange(r // 2, device="cuda", dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / s["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(s["factor"]) + 1.0
    # bands: by the number of turns, between low_freq_factor and high_freq_factor
    keep = ((turns - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])).clamp(0, 1)
    return f * keep + f / s["factor"] * (1 - keep), amp


def _plain_table(s):
    c = s["c"]
    f, amp = _plain_frequencies(c, c["rotary"])
    angle = (torch.arange(c["positions"], device="cuda", dtype=torch.float64) + s["first"])[:, None] * f
    return torch.cat([angle.cos() * amp, angle.sin() * amp], 1).to(torch.float32 if c["fp32"] else torch.bfloat16)


def _plain_rotate(x, cos, sin, r, layout):
    x = x.to(torch.float32)
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if layout == "half" else (x[..., 0:r:2], x[..., 1:r:2])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([u, v], -1) if layout == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1).to(torch.bfloat16)


def _plain_rope(s):
    c = s["c"]
    r = c["rotary"]
    rows = s["table"][s["positions"]].to(torch.float32)[:, None]
    cos, sin = rows[..., :r // 2], rows[..., r // 2:]
    if c["inverse"]:
        sin = -sin
    q, k = _plain_rotate(s["q"], cos, sin, r, c["layout"]), _plain_rotate(s["k"], cos, sin, r, c["layout"])
    if not c["insert"]:
        return {"q": q, "k": k}
    cache, slots, bs = s["cache"], s["slots"], c["block"]
    if c["fp8"]:
        code = lambda x, scale: (x.to(torch.float32) / scale).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        row = torch.cat([code(k, s["k_scale"]), code(s["v"], s["v_scale"])], -1)
    else:
        row = torch.cat([k, s["v"]], -1)
    # a padded token writes again what the token of the highest slot writes
    last = slots.argmax()
    live = slots >= 0
    at = torch.where(live, slots, slots[last])
    cache[at // bs, :, at % bs] = torch.where(live[:, None, None], row, row[last])
    return {"q": q, "k": k, "cache": cache.view(torch.float8_e4m3fn) if c["fp8"] else cache}


def _plain_rows(s, half):
    """[B, S, Hkv, D] in 32 bits: the cached K (half 0) or V (half 1) of every request, padded to the longest."""
    c = s["c"]
    j = torch.arange(s["longest"], device="cuda")
    block = s["table"][:, j // c["block"]].long().clamp(min=0)
    D = c["dim"]
    rows = s["cache"][..., half * D:(half + 1) * D][block, :, j % c["block"]]
    if c["fp8"]:
        return rows.view(torch.float8_e4m3fn).to(torch.float32) * (s["v_scale"] if half else s["k_scale"])
    return rows.to(torch.float32)


def _plain_visible(s):
    """[T, S]: which cached tokens each query sees."""
    c = s["c"]
    j = torch.arange(s["longest"], device="cuda")[None]
    ctx, of = s["ctx"].long(), s["of"]
    q = (s["start"][1:] - s["start"][:-1]).long()
    at = j - ctx[of][:, None]  # the drafted token's number, negative for the context
    drafted = (at >= 0) & (at < q[of][:, None])
    if c["mask"] == "causal":
        drafted &= at <= s["node"][:, None]
    if s["mask"] is not None:
        n = at.clamp(min=0, max=64 * s["mask"].shape[1] - 1)
        drafted &= (s["mask"].gather(1, n // 64) >> (n % 64)) & 1 == 1
    return (at < 0) | drafted


def _padded_queries(s):
    """[B, Q, H, D]: the queries, padded to the longest request."""
    c = s["c"]
    pad = torch.zeros((c["requests"], c["q_max"]) + s["q"].shape[1:], device="cuda")
    pad[s["of"], s["node"]] = s["q"].to(torch.float32)
    return pad


def _plain_scores(s):
    """([T, Hq, S] scores with -inf where a token is not seen, whether it is seen)."""
    c = s["c"]
    G = c["heads"] // c["kv_heads"]
    k = _plain_rows(s, 0).permute(0, 2, 3, 1)  # [B, Hkv, D, S]
    q = _padded_queries(s)
    B, Q, H, D = q.shape
    q = q.view(B, Q, H // G, G, D).permute(0, 2, 1, 3, 4).reshape(B, H // G, Q * G, D)
    x = torch.matmul(q, k).mul_(1.0 / math.sqrt(D))  # [B, Hkv, Q G, S]
    x = x.view(B, H // G, Q, G, -1).permute(0, 2, 1, 3, 4).reshape(B, Q, H, -1)[s["of"], s["node"]]
    seen = _plain_visible(s)[:, None]
    return x.masked_fill_(~seen, -math.inf), seen


def _plain_attention(s):
    c = s["c"]
    G = c["heads"] // c["kv_heads"]
    x, _ = _plain_scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top)[..., 0]
    p = p.div_(torch.where(total == 0, torch.ones_like(total), total))
    T, H, S = p.shape
    B, Q, D = c["requests"], c["q_max"], c["dim"]
    pad = torch.zeros((B, Q, H, S), device="cuda")
    pad[s["of"], s["node"]] = p
    del p, x
    pad = pad.view(B, Q, H // G, G, S).permute(0, 2, 1, 3, 4).reshape(B, H // G, Q * G, S)
    o = torch.matmul(pad, _plain_rows(s, 1).permute(0, 2, 1, 3))
    o = o.view(B, H // G, Q, G, D).permute(0, 2, 1, 3, 4).reshape(B, Q, H, D)[s["of"], s["node"]]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _plain_weight(s):
    c = s["c"]
    G, n = c["heads"] // c["kv_heads"], s["weights"].shape[2]
    x, _ = _plain_scores(s)
    p = x.sub_(s["lse"][..., None]).exp_()[..., :n]
    p = p.view(p.shape[0], -1, G, n).sum(2)  # [T, Hkv, S]
    total = torch.zeros_like(s["weights"]).index_add_(0, s["of"], p)
    live = (torch.arange(n, device="cuda") < s["ctx"][:, None])[:, None]
    s["weights"].copy_(torch.where(live, 0.9 * s["weights"] + total, s["weights"]))
    return {"weights": s["weights"]}


def _plain_evict(s):
    c = s["c"]
    w, pos, bs = s["weights"], s["positions"], c["block"]
    B, H, S = w.shape
    j = torch.arange(S, device="cuda")
    n = s["ctx"].long()[:, None, None]
    keep_n = n.clamp(max=c["budget"])
    key = torch.where(w.isnan(), torch.full_like(w, -math.inf), w)
    key = torch.where((pos < SINKS) | (pos >= s["seen"][:, None, None] - RECENT), torch.full_like(w, math.inf), key)
    live = j < n
    # a place beyond the length sorts behind every other
    order = torch.argsort(torch.where(live, key, torch.full_like(w, -math.inf)), dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order))
    keep = (rank < keep_n) & live
    hole, mover = ~keep & (j < keep_n), keep & (j >= keep_n)
    # the i-th mover goes to the i-th hole
    dst = torch.sort((~hole).to(torch.int32), dim=-1, stable=True)[1]
    src = torch.sort((~mover).to(torch.int32), dim=-1, stable=True)[1]
    b, h, i = torch.nonzero(j < hole.sum(-1, keepdim=True), as_tuple=True)
    d, e = dst[b, h, i], src[b, h, i]
    wo, po = s["weights_out"], s["positions_out"]
    wo.copy_(torch.where(live & (j >= keep_n), torch.zeros_like(w), w))
    po.copy_(torch.where(live & (j >= keep_n), torch.full_like(pos, -1), pos))
    wo[b, h, d], po[b, h, d] = w[b, h, e], pos[b, h, e]
    cache, t = s["cache"], s["table"].long()
    cache[t[b, d // bs], h, d % bs] = cache[t[b, e // bs], h, e % bs]
    return {"cache": cache.view(torch.float8_e4m3fn) if c["fp8"] else cache, "weights": wo, "positions": po,
            "lens": s["ctx"].clamp(max=c["budget"])}


SINKS, RECENT = 4, 16


# ------------------------------------------------------------------ one pass


def run(state):
    s = state
    if not own:
        return {"table": _plain_table, "rope": _plain_rope, "attention": _plain_attention, "weight": _plain_weight,
                "evict": _plain_evict}[s["op"]](s)
    import speculative_decoding_draft_ctx_gb300 as dk

    c = s["c"]
    if s["op"] == "table":
        return dk.rope_table(c["positions"], c["rotary"], theta=c["theta"], scaling=_scaling(c), first_position=s["first"],
                             dtype=torch.float32 if c["fp32"] else torch.bfloat16, device="cuda")
    if s["op"] == "rope":
        more = dict(v=s["v"], slot_mapping=s["slots"], kv_cache=s["cache"], k_scale=s["k_scale"], v_scale=s["v_scale"]) if c["insert"] else {}
        q, k = dk.rope_kv_insert(s["q"], s["k"], s["table"], s["positions"], c["rotary"], layout=c["layout"], inverse=c["inverse"], **more)
        if not c["insert"]:
            return {"q": q, "k": k}
        return {"q": q, "k": k, "cache": s["cache"].view(torch.float8_e4m3fn) if c["fp8"] else s["cache"]}
    if s["op"] == "attention":
        out, lse = dk.tree_attention(s["q"], s["cache"], s["table"], s["start"], s["ctx"], tree_mask=s["mask"], causal=c["mask"] == "causal",
                                     k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"out": out, "lse": lse}
    if s["op"] == "weight":
        return {"weights": dk.accumulate_attention_weight(s["q"], s["cache"], s["table"], s["start"], s["ctx"], s["lse"], s["weights"],
                                                          decay=0.9, k_scale=s["k_scale"])}
    lens = dk.evict_kv(s["cache"], s["table"], s["ctx"], s["weights"], s["positions"], s["seen"], c["budget"], sinks=SINKS, recent=RECENT,
                       weights_out=s["weights_out"], positions_out=s["positions_out"])
    return {"cache": s["cache"].view(torch.float8_e4m3fn) if c["fp8"] else s["cache"], "weights": s["weights_out"],
            "positions": s["positions_out"], "lens": lens}


# ------------------------------------------------------------------ floors


def work(case):
    c = case
    if c["op"] == "table":
        n = c["positions"] * c["rotary"]
        return {"bytes": n * (4 if c["fp32"] else 2), "flops": 10 * n}
    if c["op"] == "rope":
        T, Hq, Hk, D, r = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["rotary"]
        size = T * (Hq + Hk) * D * 4 + T * (8 + 2 * r)
        if c["insert"]:
            size += T * Hk * D * 2 + T * 8 + T * Hk * 2 * D * (1 if c["fp8"] else 2)
        return {"bytes": size, "flops": 3 * T * (Hq + Hk) * r}
    ctx, q = _lengths(c)
    H, D, e = c["kv_heads"], c["dim"], 1 if c["fp8"] else 2
    if c["op"] == "evict":
        entries = sum(ctx) * H
        moved = sum(H * min(n, c["budget"]) * (1 - min(n, c["budget"]) / n) for n in ctx if n)
        return {"bytes": int(entries * 16 + moved * 2 * 2 * D * e), "flops": entries}
    T = sum(q)
    if c["op"] == "weight":
        return {"bytes": sum(ctx) * H * (D * e + 8) + T * c["heads"] * (2 * D + 4),
                "flops": sum(2 * D * m * c["heads"] * n for n, m in zip(ctx, q))}
    total = sum(n + m for n, m in zip(ctx, q))
    return {"bytes": total * H * 2 * D * e + T * c["heads"] * (4 * D + 4),
            "flops": sum(4 * D * m * c["heads"] * (n + m) for n, m in zip(ctx, q))}


# ------------------------------------------------------------------ from the definitions, in 64 bits


def _exact_table(c, first):
    import numpy as np

    r, s = c["rotary"], _scaling(c)
    f, amp = [], 1.0
    for i in range(r // 2):
        x = c["theta"] ** (-2.0 * i / r)
        if s is not None and s["kind"] == "linear":
            x /= s["factor"]
        elif s is not None and s["kind"] == "by_parts":
            amp = 0.1 * math.log(s["factor"]) + 1.0
            edge = [r * math.log(s["original_positions"] / (t * 2 * math.pi)) / (2 * math.log(c["theta"])) for t in (s["beta_fast"], s["beta_slow"])]
            lo, hi = max(0, math.floor(edge[0])), min(r - 1, math.ceil(edge[1]))
            m = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            x = x / s["factor"] * m + x * (1 - m)
        elif s is not None:
            t = s["original_positions"] * x / (2 * math.pi)
            m = min(1.0, max(0.0, (t - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])))
            x = x * m + x / s["factor"] * (1 - m)
        f.append(x)
    a = np.arange(first, first + c["positions"], dtype=np.float64)[:, None] * np.array(f)
    return np.concatenate([np.cos(a), np.sin(a)], 1) * amp


def _exact_rope(s):
    c = s["c"]
    r, D, T = c["rotary"], c["dim"], c["tokens"]
    row = s["table"].double()[s["positions"]]
    turn = torch.complex(row[:, :r // 2], row[:, r // 2:] * (-1 if c["inverse"] else 1))[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        first = torch.arange(r // 2, device="cuda") * (1 if c["layout"] == "half" else 2)
        second = first + (r // 2 if c["layout"] == "half" else 1)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    if not c["insert"]:
        return out
    cache = s["cache"].view(torch.float8_e4m3fn).double() if c["fp8"] else s["cache"].double()
    k, v = out["k"].to(torch.bfloat16).double(), s["v"].double()
    if c["fp8"]:
        k, v = (k / s["k_scale"].double()).clamp(-FP8_MAX, FP8_MAX), (v / s["v_scale"].double()).clamp(-FP8_MAX, FP8_MAX)
    live = s["slots"] >= 0
    at = s["slots"][live]
    cache[at // c["block"], :, at % c["block"]] = torch.cat([k, v], -1)[live]
    return {**out, "cache": cache}


def _exact_request(s, b):
    """Request b's queries [Q, H, D], keys and values [S, Hkv, D] in 64 bits, and its lengths."""
    c = s["c"]
    lo, hi, n = int(s["start"][b]), int(s["start"][b + 1]), int(s["ctx"][b])
    m = n + hi - lo
    j = torch.arange(m, device="cuda")
    raw = s["cache"][s["table"][b].long()[j // c["block"]], :, j % c["block"]]
    D = c["dim"]
    if c["fp8"]:
        rows = raw.view(torch.float8_e4m3fn).double()
        k, v = rows[..., :D] * s["k_scale"].double(), rows[..., D:] * s["v_scale"].double()
    else:
        k, v = raw[..., :D].double(), raw[..., D:].double()
    return lo, hi, n, s["q"][lo:hi].double(), k, v


def _exact_seen(s, lo, hi, n):
    """[Q, S] truth values of one request."""
    Q, c = hi - lo, s["c"]
    tail = torch.ones((Q, Q), dtype=torch.bool, device="cuda")
    if c["mask"] == "causal":
        tail = tail.tril()
    if s["mask"] is not None:
        i = torch.arange(Q, device="cuda")
        tail = torch.stack([(s["mask"][lo:hi, int(j) // 64] >> (int(j) % 64)) & 1 for j in i.tolist()], 1).bool()
    return torch.cat([torch.ones((Q, n), dtype=torch.bool, device="cuda"), tail], 1)


def _exact_heads(q, k, c, h):
    """Scores of KV head h: [Q, G, S]."""
    G = c["heads"] // c["kv_heads"]
    return (q[:, h * G:(h + 1) * G] @ k[:, h].T) * c["dim"] ** -0.5


def _exact_attention(s):
    c = s["c"]
    G = c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["requests"]):
        lo, hi, n, q, k, v = _exact_request(s, b)
        if hi == lo:
            continue
        seen = _exact_seen(s, lo, hi, n)[:, None]
        for h in range(c["kv_heads"]):
            x = _exact_heads(q, k, c, h).masked_fill(~seen, -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.where(z[..., None] == -math.inf, torch.zeros_like(x), (x - z[..., None]).exp())
            out[lo:hi, h * G:(h + 1) * G] = p @ v[:, h]
            lse[lo:hi, h * G:(h + 1) * G] = z
    return {"out": out, "lse": lse}


def _exact_weight(s):
    c = s["c"]
    G = c["heads"] // c["kv_heads"]
    w = s["weights"].double()
    for b in range(c["requests"]):
        lo, hi, n, q, k, _ = _exact_request(s, b)
        for h in range(c["kv_heads"]):
            x = _exact_heads(q, k[:n], c, h) - s["lse"][lo:hi, h * G:(h + 1) * G, None].double()
            w[b, h, :n] = 0.9 * w[b, h, :n] + x.exp().sum((0, 1))
    return {"weights": w}


def _exact_evict(s):
    import numpy as np

    c = s["c"]
    w, pos, ctx = s["weights"].cpu().numpy(), s["positions"].cpu().numpy(), s["ctx"].cpu().numpy()
    table, seen = s["table"].cpu().numpy(), s["seen"].cpu().numpy()
    wo, po = w.copy(), pos.copy()
    moves = []
    for b in range(w.shape[0]):
        n = int(ctx[b])
        k = min(n, c["budget"])
        if n <= k:
            continue
        for h in range(w.shape[1]):
            key = np.where(np.isnan(w[b, h, :n]), -np.inf, w[b, h, :n])
            key[(pos[b, h, :n] < SINKS) | (pos[b, h, :n] >= seen[b] - RECENT)] = np.inf
            kept = np.sort(np.argsort(-key, kind="stable")[:k])
            src = kept[kept >= k]
            dst = np.setdiff1d(np.arange(k), kept[kept < k], assume_unique=True)
            wo[b, h, k:n], po[b, h, k:n] = 0.0, -1
            wo[b, h, dst], po[b, h, dst] = w[b, h, src], pos[b, h, src]
            at = lambda j: (table[b, j // c["block"]].astype(np.int64) * w.shape[1] + h) * c["block"] + j % c["block"]  # noqa: E731,B023
            moves.append((at(dst), at(src)))
    cache = s["cache"].view(torch.float8_e4m3fn) if c["fp8"] else s["cache"]
    flat = s["cache"].view(-1, 2 * c["dim"])
    if moves:
        to, of = (torch.from_numpy(np.concatenate([m[i] for m in moves])).cuda() for i in (0, 1))
        flat[to] = flat[of]
    return {"cache": cache, "weights": torch.from_numpy(wo).double(), "positions": torch.from_numpy(po),
            "lens": torch.from_numpy(np.minimum(ctx, c["budget"]))}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "table":
        return _exact_table(s["c"], s["first"])
    if s["op"] == "rope":
        return _exact_rope(s)
    return {"attention": _exact_attention, "weight": _exact_weight, "evict": _exact_evict}[s["op"]](s)
