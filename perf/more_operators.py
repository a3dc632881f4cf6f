"""Measured cases of the operators around a draft step's verification.

Each case is one pass as a serving loop makes it: the verification of drafted
tokens against the target's probabilities (``verify``), the accepted path's
K/V moved behind the context in every layer (``compact``), pages of a pool
shared, copied, reserved and freed (``pages``), the insert into a cache of
8-bit codes with one power-of-two scale per page and head (``insert``) and the
attention over such a cache (``attention``).  ``own`` false computes the plain
form in elementary torch operations; true makes the framework's calls.
"""

import math
import random

import torch

own = False

FP8_MAX = 448.0
EXP_MIN, EXP_MAX = -32, 31  # a page's scale is a power of two from this range


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one request's chain of seven drafted tokens (latency)
        dict(name="verify_one", op="verify", requests=1, n_min=7, n_max=7, vocab=32000, tree=1, draft="probs", replacement=True, bf16=False),
        # a serving batch's chains
        dict(name="verify_serving", op="verify", requests=64, n_min=7, n_max=7, vocab=131072, tree=1, draft="probs", replacement=True, bf16=False),
        # trees of up to 63 drafted tokens, children drawn without replacement, an odd vocabulary
        dict(name="verify_trees", op="verify", requests=12, n_min=15, n_max=63, vocab=100003, tree=4, draft="probs", replacement=False, bf16=False),
        # one request's accepted path, five layers (latency)
        dict(name="compact_one", op="compact", requests=1, n_min=63, n_max=63, accept=6, layers=5, kv_heads=8, dim=128, block=16, kind="bf16"),
        # a serving batch of trees over the 8-bit cache
        dict(name="compact_serving", op="compact", requests=64, n_min=31, n_max=63, accept=7, layers=5, kv_heads=8, dim=128, block=16, kind="scaled"),
        # one prompt answered four times: its last page copied, pages for the next step
        dict(name="pages_one", op="pages", live=1, forks=3, finished=0, ctx_min=300, ctx_max=300, draft=8, pool=512, layers=5, kv_heads=8, dim=128, block=64, kind="bf16"),
        # a serving batch: 16 prompts forked, others finished, everyone's next pages from a large pool
        dict(name="pages_serving", op="pages", live=96, forks=64, finished=32, ctx_min=256, ctx_max=8192, draft=64, pool=65536, layers=2, kv_heads=4, dim=128, block=16, kind="scaled"),
        # a draft step's tokens of 64 requests
        dict(name="insert_step", op="insert", requests=64, q_min=1, q_max=7, ctx_min=1024, ctx_max=8192, kv_heads=8, dim=128, block=16),
        # a prefill batch
        dict(name="insert_prefill", op="insert", requests=32, q_min=256, q_max=256, ctx_min=0, ctx_max=0, kv_heads=8, dim=128, block=64),
        # one request's single token (latency)
        dict(name="attn_scaled_one", op="attention", requests=1, q_min=1, q_max=1, heads=64, kv_heads=8, dim=128, ctx_min=300, ctx_max=300, block=16, mask="dense"),
        # a draft step of 64 requests
        dict(name="attn_scaled_step", op="attention", requests=64, q_min=7, q_max=7, heads=64, kv_heads=8, dim=128, ctx_min=1024, ctx_max=8192, block=16, mask="causal"),
        # trees over two long contexts
        dict(name="attn_scaled_long", op="attention", requests=2, q_min=40, q_max=64, heads=32, kv_heads=4, dim=128, ctx_min=65537, ctx_max=131072, block=128, mask="tree"),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["verify", "verify", "compact", "pages", "insert", "attention", "attention"])
    dim = rng.choice([64, 128, 128, 256])
    block = rng.choice([1, 3, 16, 16, 32, 48, 64, 100, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    kind = rng.choice(["bf16", "fp8", "scaled"])
    if op == "verify":
        tree = rng.choice([1, 1, 2, 4])
        n = _log(rng, 1, 63 if tree > 1 else 31)
        vocab = _log(rng, 1000, 131072)
        requests = _log(rng, 1, max(1, min(64, 64 * 8 * 131072 // ((n + 1) * vocab), 12 * 64 * 100003 // ((n + 1) * vocab) if tree > 1 else 64)))
        return dict(op=op, requests=requests, n_min=rng.randint(1, n), n_max=n, vocab=vocab, tree=tree,
                    draft=rng.choice(["probs", "probs", "none"]), replacement=rng.random() < 0.5, bf16=rng.random() < 0.3)
    if op == "compact":
        n = _log(rng, 2, 63)
        return dict(op=op, requests=_log(rng, 1, 64), n_min=rng.randint(2, n), n_max=n, accept=rng.randint(1, 12), layers=rng.randint(1, 5),
                    kv_heads=kv_heads, dim=dim, block=block, kind=kind)
    if op == "pages":
        live = _log(rng, 1, 96)
        forks = _log(rng, 1, 64)
        finished = rng.randint(0, live - 1)
        block = max(block, 16)
        ctx = _log(rng, 20, 4096)
        pool = (live + forks + 2) * (ctx // block + 8)
        pool = min(pool + rng.randint(0, pool), (1 << 29) // (min(kv_heads, 4) * block * dim))
        return dict(op=op, live=live, forks=forks, finished=finished, ctx_min=rng.randint(1, ctx), ctx_max=ctx, draft=rng.randint(1, 64),
                    pool=pool, layers=rng.randint(1, 2), kv_heads=min(kv_heads, 4), dim=dim, block=block, kind=kind)
    if op == "insert":
        requests = _log(rng, 1, 64)
        q = _log(rng, 1, max(1, min(256, 8192 * 1024 // (requests * kv_heads * dim))))
        ctx = _log(rng, 1, 8192)
        return dict(op=op, requests=requests, q_min=rng.randint(1, q), q_max=q, ctx_min=rng.choice([0, ctx // 2]), ctx_max=ctx,
                    kv_heads=kv_heads, dim=dim, block=block)
    requests = _log(rng, 1, 64)
    group = rng.choice([1, 2, 3, 5, 8, 16])
    q_max = rng.choice([1, _log(rng, 1, 64)])
    rows = q_max * group * kv_heads
    longest = min(131072, (1 << 28) // (requests * kv_heads * dim), (1 << 29) // (requests * rows))
    ctx = _log(rng, 1, max(64, longest))
    return dict(op=op, requests=requests, q_min=rng.randint(1, q_max), q_max=q_max, heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                ctx_min=rng.choice([1, ctx // 2 + 1]), ctx_max=ctx, block=block, mask=rng.choice(["dense", "causal", "tree"]))


def _spread(n, lo, hi, step):
    """n whole numbers over [lo, hi], over their logarithm: the same ones each time, the first the largest."""
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [hi if i == 0 else min(hi, max(lo, int(round(math.exp(b - (b - a) * ((i * step) % 1.0)) - 1)))) for i in range(n)]


def _lengths(c):
    """Context tokens and new tokens of every request."""
    ctx = _spread(c["requests"], c["ctx_min"], c["ctx_max"], 0.618034)
    return ctx, _spread(c["requests"], c["q_min"], c["q_max"], 0.414214)


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _drafts(c):
    """Drafted tokens of every request of a verification or a compaction."""
    return _spread(c["requests"], c["n_min"], c["n_max"], 0.414214)


def _depth(c):
    return c["n_max"] if c["tree"] == 1 else min(c["n_max"], 8)


# ------------------------------------------------------------------ inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _block_table(block, need, g, width=None):
    """Every request's shuffled physical blocks, and how many blocks there are."""
    held = [-(-n // block) for n in need]
    count = sum(held)
    order = torch.randperm(count + 3, generator=g, device="cuda")[:count].to(torch.int32).cpu()
    table = torch.full((len(need), width or max(1, max(held))), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(held):
        table[b, :m] = order[at:at + m]
        at += m
    return table.cuda(), count + 3


def _caches(c, blocks, g, layers):
    """(layers' caches with every slot written, their page scales or None)."""
    shape = (blocks, c["kv_heads"], c["block"], 2 * c["dim"])
    kind, caches, scales = c.get("kind", "scaled"), [], []
    for _ in range(layers):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        if kind == "bf16":
            caches.append(x)
            continue
        # values of a page and head spread over their scale's range
        caches.append((x * 100).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8))
        scales.append(torch.randint(-8, -4, (blocks, c["kv_heads"], 2), generator=g, device="cuda", dtype=torch.int8))
    return caches, scales if kind == "scaled" else None


def _parents(n, arity, rnd):
    """Parent rows of rows 0 .. n of a tree with up to `arity` children a row (row 0: the token behind which it grows)."""
    if arity == 1:
        return [-1] + list(range(n))
    parents, kids, depth = [-1], [0], [0]
    for i in range(1, n + 1):
        # breadth comes first near the root, as a drafter's beams grow
        open_rows = [r for r in range(i) if kids[r] < arity and depth[r] < 8]
        p = open_rows[min(int(rnd.expovariate(0.35)), len(open_rows) - 1)]
        parents.append(p)
        kids.append(0)
        depth.append(depth[p] + 1)
        kids[p] += 1
    return parents


def _prepare_verify(c, g, seed):
    rnd, drafts, V = random.Random(seed), _drafts(c), c["vocab"]
    start = _starts([n + 1 for n in drafts])
    T = start[-1]
    # a target's distributions: heavy heads and long tails; every other request's cut off at a share of the largest, as sampling does
    target = torch.randn((T, V), generator=g, device="cuda").mul_(4)
    draft = None
    if c["draft"] == "probs":
        draft = torch.randn((T, V), generator=g, device="cuda").mul_(0.8).add_(target, alpha=0.95)
        draft.sub_(draft.amax(1, keepdim=True)).exp_()
        draft.div_(draft.sum(1, keepdim=True))
    target.sub_(target.amax(1, keepdim=True)).exp_()
    of = torch.repeat_interleave(torch.arange(len(drafts), device="cuda"), _ints([n + 1 for n in drafts], torch.int64))
    target.masked_fill_((target < 1e-4) & (of % 2 == 1)[:, None], 0.0)
    target.div_(target.sum(1, keepdim=True))
    if c["bf16"]:
        target = target.to(torch.bfloat16)
        draft = None if draft is None else draft.to(torch.bfloat16)
    parents = [p for n in drafts for p in _parents(n, c["tree"], rnd)]
    # the k-th child of a row: the k-th in the order of log q + noise (without replacement), or a draw of its own
    base = draft if draft is not None else target
    tokens = torch.zeros(T, dtype=torch.int64, device="cuda")
    rank, rows, up = [0] * T, [], []
    for b, n in enumerate(drafts):
        kids = {}
        for i in range(1, n + 1):
            t, p = start[b] + i, parents[start[b] + i]
            rank[t] = kids.get(p, 0)
            kids[p] = rank[t] + 1
            rows.append(t)
            up.append(start[b] + p)
    rows, up, ranks = _ints(rows, torch.int64), _ints(up, torch.int64), _ints([rank[t] for t in rows], torch.int64)
    if c["replacement"] and c["draft"] == "probs":
        for lo in range(0, len(rows), 64):  # by the inverse of the cumulated probabilities
            cum = base[up[lo:lo + 64]].to(torch.float64).cumsum(1)
            u = torch.rand((len(cum), 1), generator=g, device="cuda", dtype=torch.float64) * cum[:, -1:]
            tokens[rows[lo:lo + 64]] = (cum <= u).sum(1).clamp(max=V - 1)
    else:
        for lo in range(0, T, 64):
            x = base[lo:lo + 64].to(torch.float32).log()
            if c["draft"] == "probs":
                x -= torch.empty_like(x).exponential_(generator=g).log_()
            top = x.topk(c["tree"], dim=1)[1]
            here = (up >= lo) & (up < lo + 64)
            tokens[rows[here]] = top[up[here] - lo, ranks[here]]
    return dict(op="verify", c=c, target=target, draft=draft, tokens=tokens, start=_ints(start), parents=_ints(parents) if c["tree"] > 1 else None,
                uniforms=torch.rand(T, generator=g, device="cuda"), drafts=drafts)


def _prepare_compact(c, g, seed):
    rnd, drafts = random.Random(seed), _drafts(c)
    ctx = _spread(len(drafts), 20, 1000, 0.618034)
    table, blocks = _block_table(c["block"], [n + 1 + m for n, m in zip(ctx, drafts)], g)
    caches, scales = _caches(c, blocks, g, c["layers"])
    if scales is not None:
        # the drafted tokens were inserted in one step: their pages behind the context's last have one scale
        tail = table.clamp(min=0).long()
        behind = torch.arange(table.shape[1], device="cuda") > (_ints(ctx) // c["block"])[:, None]
        behind &= table >= 0
        last = tail.gather(1, (_ints(ctx, torch.int64) // c["block"])[:, None]).expand_as(tail)
        step = (2 * (torch.arange(len(ctx), device="cuda") % 2) - 1)[:, None].expand_as(tail)[behind]
        for x in scales:
            x[tail[behind]] = x[last[behind]] + step[:, None, None].to(x.dtype)
    rows = torch.full((len(drafts), c["accept"]), -1, dtype=torch.int32)
    counts = []
    for b, n in enumerate(drafts):
        # the path keeps to the first branch for a while, then leaves it for rows behind everything that it moves to
        k = rnd.randint(0, min(c["accept"], n // 2))
        stay = rnd.randint(0, k)
        path = list(range(1, stay + 1)) + sorted(rnd.sample(range(k + 1, n + 1), k - stay))
        rows[b, :k] = torch.tensor(path, dtype=torch.int32)
        counts.append(k)
    return dict(op="compact", c=c, caches=caches, scales=scales, table=table, ctx=_ints(ctx), rows=rows.cuda(), counts=_ints(counts))


def _prepare_pages(c, g, seed):
    rnd, bs = random.Random(seed), c["block"]
    R = c["live"] + c["forks"]
    lens = _spread(c["live"], c["ctx_min"], c["ctx_max"], 0.618034)
    width = -(-(c["ctx_max"] + c["draft"]) // bs) + 1
    held = [-(-n // bs) for n in lens]
    while sum(held) + c["forks"] + R * (-(-c["draft"] // bs) + 1) > c["pool"]:  # the pool holds what the step asks for
        lens = [max(1, n // 2) for n in lens]
        held = [-(-n // bs) for n in lens]
    order = torch.randperm(c["pool"], generator=g, device="cuda")[:sum(held)].to(torch.int32).cpu()
    table, refs = torch.full((R, width), -1, dtype=torch.int32), torch.zeros(c["pool"], dtype=torch.int32)
    rows = list(range(R))
    rnd.shuffle(rows)  # rows of live requests and free ones in no order
    live, free = rows[:c["live"]], rows[c["live"]:]
    pages, tokens, at = [0] * R, [0] * R, 0
    for r, n, m in zip(live, lens, held):
        table[r, :m] = order[at:at + m]
        refs[order[at:at + m].long()] = 1
        pages[r], tokens[r] = m, n
        at += m
    sources = live[c["finished"]:]
    keep = [1] * R
    for r in live[:c["finished"]]:
        keep[r] = 0
    caches, scales = _caches(c, c["pool"], g, c["layers"])
    return dict(op="pages", c=c, caches=caches, scales=scales, src=_ints([sources[i % min(16, len(sources))] for i in range(c["forks"])]), dst=_ints(free),
                keep=_ints(keep) == 1, held=dict(table=table.cuda(), refs=refs.cuda(), pages=_ints(pages), lens=_ints(tokens)),
                # what the step works on; a pass starts from `held` again
                table=table.cuda(), refs=refs.cuda(), pages=_ints(pages), lens=_ints(tokens))


def _tree_masks(q, words, seed):
    """Bit j of row i: node j is node i or one of its ancestors."""
    r, rows = random.Random(seed), []
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
    if c["op"] == "verify":
        return _prepare_verify(c, g, seed)
    if c["op"] == "compact":
        return _prepare_compact(c, g, seed)
    if c["op"] == "pages":
        return _prepare_pages(c, g, seed)
    ctx, q = _lengths(c)
    table, blocks = _block_table(c["block"], [n + m for n, m in zip(ctx, q)], g)
    caches, scales = _caches(c, blocks, g, 1)
    T, D = sum(q), c["dim"]
    s = dict(op=c["op"], c=c, cache=caches[0], scales=scales[0], table=table, ctx=_ints(ctx), start=_ints(_starts(q)),
             longest=max(n + m for n, m in zip(ctx, q)), of=_ints([b for b, m in enumerate(q) for _ in range(m)], torch.int64),
             node=_ints([i for m in q for i in range(m)], torch.int64))
    if c["op"] == "insert":
        kv = torch.randn((T, 2 * c["kv_heads"], D), generator=g, device="cuda", dtype=torch.bfloat16)
        kv *= torch.rand((T, 1, 1), generator=g, device="cuda").mul_(4).exp_().to(torch.bfloat16)  # tokens of unlike size
        s["k"], s["v"] = kv[:, :c["kv_heads"]], kv[:, c["kv_heads"]:]
        return s
    s["q"] = torch.randn((T, c["heads"], D), generator=g, device="cuda", dtype=torch.bfloat16)
    s["mask"] = _tree_masks(q, -(-c["q_max"] // 64), seed) if c["mask"] == "tree" else None
    return s


# ------------------------------------------------------------------ plain forms


def _plain_verify(s):
    """The walk from the root in every request at once, in 64 bits: r = max(p - S q, 0) is what rejections leave of p."""
    c, V = s["c"], s["c"]["vocab"]
    target, draft, tokens = s["target"], s["draft"], s["tokens"]
    start = s["start"].long()
    T, B, dev = tokens.numel(), start.numel() - 1, tokens.device
    t = torch.arange(T, device=dev)
    of = torch.searchsorted(start[1:], t, right=True)
    first = start[of]
    local = t - first
    up = torch.where(local > 0, first + (local - 1 if s["parents"] is None else s["parents"].long()), torch.full_like(t, -1))
    # kids[t, k]: the k-th child of row t
    same = (up[:, None] == up[None]) & (up >= 0)[:, None]
    rank = (same & (t[None] < t[:, None])).sum(1)
    kids = torch.full((T, c["tree"]), -1, dtype=torch.int64, device=dev)
    kid = local > 0
    kids.index_put_((up.clamp(min=0), torch.where(kid, rank, torch.zeros_like(rank))), torch.where(kid, t + 1, torch.zeros_like(t)), accumulate=True)
    kids = torch.where(kids >= 0, kids, torch.full_like(kids, -1))
    depth = _depth(c)
    out_tokens = torch.full((B, depth + 1), -1, dtype=torch.int64, device=dev)
    out_rows = torch.full((B, depth), -1, dtype=torch.int32, device=dev)
    cur, count = start[:-1].clone(), torch.zeros(B, dtype=torch.int64, device=dev)
    going = torch.ones(B, dtype=torch.bool, device=dev)
    S, Q = (torch.zeros(B, dtype=torch.float64, device=dev) for _ in range(2))  # S, and the rejected children's share of q
    gone = torch.full((B, c["tree"]), -1, dtype=torch.int64, device=dev)  # the rejected children's tokens
    req = torch.arange(B, device=dev)

    def rest(mass_only):
        p = target[cur].double()
        if draft is not None:
            r = (p - S[:, None] * draft[cur].double()).clamp_(min=0)
        else:
            r = p.clone()
            hit = torch.zeros((B, V + 1), dtype=torch.bool, device=dev)
            hit.scatter_(1, torch.where(gone >= 0, gone, torch.full_like(gone, V)), True)
            r.masked_fill_(hit[:, :V], 0.0)
        if mass_only:
            return r.sum(1)
        # nothing left: the target's own distribution
        return torch.where((r.sum(1) > 0)[:, None], r, p)

    for d in range(depth):
        Z = torch.ones_like(S)
        testing, taken = going.clone(), torch.zeros_like(going)
        nxt = cur.clone()
        for k in range(c["tree"]):
            child = kids[cur, k]
            testing &= (child >= 0) & ~taken
            at = child.clamp(min=0)
            x, u = tokens[at], s["uniforms"][at].double()
            p = target[cur, x].double()
            if draft is not None:
                if k:
                    Z = torch.where(testing, rest(True), Z)
                left = (1 - Q) if not c["replacement"] else torch.ones_like(Q)
                testing &= (left > 2.0 ** -24) & (Z > 0)
                q = draft[cur, x].double() / left.clamp(min=2.0 ** -24)
                take = testing & (u * q * Z < (p - S * draft[cur, x].double()).clamp(min=0))
                lose = testing & ~take
                S = torch.where(lose, S + Z / left.clamp(min=2.0 ** -24), S)
                Q = torch.where(lose, Q + draft[cur, x].double(), Q)
            else:
                p = torch.where((gone == x[:, None]).any(1), torch.zeros_like(p), p)
                testing &= Z > 0
                take = testing & (u * Z < p)
                lose = testing & ~take
                Z = torch.where(lose, Z - p, Z)
                gone[:, k] = torch.where(lose, x, gone[:, k])
            nxt = torch.where(take, at, nxt)
            taken |= take
        going = taken
        out_tokens[req, d] = torch.where(taken, tokens[nxt], out_tokens[req, d])
        out_rows[req, d] = torch.where(taken, (nxt - start[:-1]).to(torch.int32), out_rows[req, d])
        count += taken
        cur = nxt
        # where the path ends, what its last row's rejections left stays
        S, Q = torch.where(taken, torch.zeros_like(S), S), torch.where(taken, torch.zeros_like(Q), Q)
        gone = torch.where(taken[:, None], torch.full_like(gone, -1), gone)
    cum = rest(False).cumsum(1)
    level = s["uniforms"][start[:-1]].double() * cum[:, -1]
    last = torch.searchsorted(cum, cum[:, -1:].contiguous()).squeeze(1)  # the last with any weight
    token = torch.minimum((cum <= level[:, None]).sum(1), last)
    out_tokens[req, count] = token
    return {"tokens": out_tokens, "rows": out_rows, "counts": count.to(torch.int32)}


def _dequantised(codes, scales):
    """Codes [..., 2 D] with exponents [..., 2] of K and of V, in 32 bits."""
    D = codes.shape[-1] // 2
    return codes.view(torch.float8_e4m3fn).to(torch.float32) * torch.exp2(scales.to(torch.float32)).repeat_interleave(D, -1)


def _codes(x, exponents):
    """x / 2^exponents (of K and V in the last dim) as e4m3 codes."""
    D = x.shape[-1] // 2
    y = x * torch.exp2(-exponents.to(torch.float32)).repeat_interleave(D, -1)
    return y.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _view(s, cache):
    return cache.view(torch.float8_e4m3fn) if cache.dtype is torch.uint8 else cache


def _plain_compact(s):
    c, bs, first = s["c"], s["c"]["block"], 1
    rows, counts, ctx, table = s["rows"].long(), s["counts"].long(), s["ctx"].long(), s["table"].long()
    B, W = rows.shape
    j = torch.arange(W, device=rows.device)
    live = j < counts[:, None]
    src, dst = ctx[:, None] + torch.where(live, rows, torch.zeros_like(rows)), ctx[:, None] + first + j
    live &= src != dst
    # a place that does not move writes its own rows again: the token's that the request's path grows behind
    src, dst = torch.where(live, src, ctx[:, None]), torch.where(live, dst, ctx[:, None])
    b = torch.arange(B, device=rows.device)[:, None]
    sp, so, dp, do = table[b, src // bs], src % bs, table[b, dst // bs], dst % bs
    for layer, cache in enumerate(s["caches"]):
        if s["scales"] is None:
            cache[dp, :, do] = cache[sp, :, so]
            continue
        scales = s["scales"][layer]
        moved = _dequantised(cache[sp, :, so], scales[sp])  # [B, W, H, 2 D]
        # a page's scale grows to the largest that comes into it; what it holds is encoded anew
        page = dp.reshape(-1)
        grown = scales.to(torch.int32).scatter_reduce(0, page[:, None, None].expand(-1, *scales.shape[1:]),
                                                       scales[sp].reshape(-1, *scales.shape[1:]).to(torch.int32), "amax")
        # the places of these pages that hold tokens after the move: all before its end
        held = cache[page]  # [B W, H, bs, 2 D]
        cache[page] = torch.where((grown[page] > scales[page]).repeat_interleave(c["dim"], -1)[:, :, None],
                                  _codes(_dequantised(held, scales[page][:, :, None]), grown[page][:, :, None]), held)
        cache[dp, :, do] = _codes(moved, grown[dp])
        scales.copy_(grown)
    out = {"lens": (ctx + first + counts).to(torch.int32), "caches": [_view(s, x) for x in s["caches"]]}
    if s["scales"] is not None:
        out["scales"] = s["scales"]
    return out


def _restore(s):
    for k, x in s["held"].items():
        s[k].copy_(x)


def _free_in_order(refs, n):
    """The n lowest numbers of pages that nobody holds, -1 behind the last."""
    free = refs == 0
    out = torch.full((n + 1,), -1, dtype=torch.int64, device=refs.device)
    at = torch.where(free, free.cumsum(0) - 1, torch.full_like(refs, n).long()).clamp(max=n)
    out.scatter_(0, at, torch.arange(refs.numel(), device=refs.device))
    return out[:n]


def _plain_pages(s):
    c, bs = s["c"], s["c"]["block"]
    _restore(s)
    table, refs, pages, lens = s["table"], s["refs"], s["pages"], s["lens"]
    src, dst = s["src"].long(), s["dst"].long()
    n = lens[src].long()
    count, tail = -(-n // bs), n % bs
    # full pages are shared, a last page that is not full is copied into a free one
    new = _free_in_order(refs, src.numel())
    order = (tail > 0).cumsum(0) - 1
    fresh = torch.where(tail > 0, new[order.clamp(min=0)], torch.full_like(n, -1))
    j = torch.arange(table.shape[1], device=table.device)
    row = torch.where(j < (n // bs)[:, None], table[src], torch.full_like(table[src], -1))
    shared = torch.zeros(refs.numel() + 1, dtype=refs.dtype, device=refs.device)
    shared.index_add_(0, torch.where(row >= 0, row, torch.full_like(row, refs.numel())).reshape(-1).long(), torch.ones(row.numel(), dtype=refs.dtype, device=refs.device))
    refs += shared[:-1]
    row = torch.where((j == (n // bs)[:, None]) & (tail > 0)[:, None], fresh.to(torch.int32)[:, None], row)
    table[dst] = torch.where(j < count[:, None], row, table[dst])
    refs.index_put_((torch.where(fresh >= 0, fresh, new[0].expand_as(fresh)),), (fresh >= 0).to(refs.dtype), accumulate=True)
    old = table[src, torch.where(tail > 0, n // bs, torch.zeros_like(n))].long()
    i = torch.arange(bs, device=table.device)
    copied = (i < tail[:, None])[:, None, :, None]
    to, of = torch.where(tail > 0, fresh, old), old  # where nothing is copied, a page that is held keeps what it holds
    for layer, cache in enumerate(s["caches"]):
        cache[to] = torch.where(copied | (tail == 0)[:, None, None, None], cache[of], cache[to])
        if s["scales"] is not None:
            s["scales"][layer][to] = s["scales"][layer][of]
    pages[dst], lens[dst] = count.to(torch.int32), n.to(torch.int32)
    # the finished requests' pages come free, everyone else's next tokens get theirs
    want = torch.where(s["keep"], lens + c["draft"], torch.zeros_like(lens)).long()
    want = torch.where(lens > 0, want, torch.zeros_like(want))
    have, need = pages.long(), -(-want // bs)
    out = (j >= need[:, None]) & (j < have[:, None])
    less = torch.zeros(refs.numel() + 1, dtype=refs.dtype, device=refs.device)
    less.index_add_(0, torch.where(out, table, torch.full_like(table, refs.numel())).reshape(-1).long(), torch.ones(table.numel(), dtype=refs.dtype, device=refs.device))
    refs -= less[:-1]
    table.masked_fill_(out, -1)
    more = (need - have).clamp(min=0)
    before = more.cumsum(0) - more
    new = _free_in_order(refs, table.numel() if table.numel() < refs.numel() else refs.numel())
    in_row = (j >= have[:, None]) & (j < need[:, None])
    which = (before[:, None] + j - have[:, None]).clamp(min=0, max=new.numel() - 1)
    table.copy_(torch.where(in_row, new[which].to(torch.int32), table))
    took = torch.zeros(refs.numel() + 1, dtype=refs.dtype, device=refs.device)
    took.index_add_(0, torch.where(in_row, table, torch.full_like(table, refs.numel())).reshape(-1).long(), torch.ones(table.numel(), dtype=refs.dtype, device=refs.device))
    refs += took[:-1]
    pages.copy_(need)
    return _pages_out(s)


def _pages_out(s):
    out = {"table": s["table"], "refs": s["refs"], "pages": s["pages"], "lens": s["lens"], "caches": [_view(s, x) for x in s["caches"]]}
    if s["scales"] is not None:
        out["scales"] = s["scales"]
    return out


def _exponents(top):
    """The least e with top <= 448 * 2^e, kept to the range of a scale."""
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(top > 0, e, torch.full_like(e, EXP_MIN)).clamp(EXP_MIN, EXP_MAX)


def _plain_insert(s):
    c, bs = s["c"], s["c"]["block"]
    cache, scales, table = s["cache"], s["scales"], s["table"].long()
    place = s["ctx"].long()[s["of"]] + s["node"]
    page, off = table[s["of"], place // bs], place % bs
    x = torch.cat([s["k"], s["v"]], -1).to(torch.float32)  # [T, H, 2 D]
    D = c["dim"]
    e = _exponents(x.abs().view(*x.shape[:2], 2, D).amax(-1)).to(torch.int32)
    # a page that held tokens keeps its scale or grows it; one that begins takes the new tokens' alone
    begun = s["ctx"].long() % bs > 0
    head = table[torch.arange(len(begun), device=table.device), (s["ctx"].long() // bs).clamp(max=table.shape[1] - 1)].clamp(min=0)
    fresh = torch.full(scales.shape, EXP_MIN, dtype=torch.int32, device=scales.device)
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=scales.device)
    touched[page] = True
    old = torch.zeros(scales.shape[0], dtype=torch.int32, device=scales.device)
    old.scatter_reduce_(0, head, torch.where(begun, s["ctx"].long() % bs, torch.zeros_like(head)).to(torch.int32), "amax")
    old = torch.where(touched, old, torch.full_like(old, bs))
    grown = torch.where((old > 0)[:, None, None], scales.to(torch.int32), fresh)
    grown = grown.scatter_reduce(0, page[:, None, None].expand_as(e), e, "amax")
    # the tokens that a growing page held are encoded anew
    held = cache[head]
    change = (begun & touched[head])[:, None, None, None] & (torch.arange(bs, device=cache.device) < (s["ctx"].long() % bs)[:, None])[:, None, :, None]
    cache[head] = torch.where(change & (grown[head] > scales[head]).repeat_interleave(D, -1)[:, :, None],
                              _codes(_dequantised(held, scales[head][:, :, None]), grown[head][:, :, None]), held)
    cache[page, :, off] = _codes(x, grown[page])
    scales.copy_(grown)
    return {"cache": cache.view(torch.float8_e4m3fn), "scales": scales}


def _plain_rows(s, half):
    """[B, S, Hkv, D] in 32 bits: the cached K (half 0) or V (half 1) of every request, padded to the longest."""
    c, D = s["c"], s["c"]["dim"]
    j = torch.arange(s["longest"], device="cuda")
    block = s["table"][:, j // c["block"]].long().clamp(min=0)
    rows = s["cache"][..., half * D:(half + 1) * D][block, :, j % c["block"]].view(torch.float8_e4m3fn).to(torch.float32)
    return rows * torch.exp2(s["scales"][..., half].to(torch.float32))[block][..., None]


def _plain_attention(s):
    c = s["c"]
    G, H, D, B, Q = c["heads"] // c["kv_heads"], c["heads"], c["dim"], c["requests"], c["q_max"]
    q = torch.zeros((B, Q, H, D), device="cuda")
    q[s["of"], s["node"]] = s["q"].to(torch.float32)
    q = q.view(B, Q, H // G, G, D).permute(0, 2, 1, 3, 4).reshape(B, H // G, Q * G, D)
    x = torch.matmul(q, _plain_rows(s, 0).permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(D))  # [B, Hkv, Q G, S]
    j = torch.arange(s["longest"], device="cuda")[None]
    ctx, of = s["ctx"].long(), s["of"]
    at = j - ctx[of][:, None]  # the drafted token's number, negative for the context
    drafted = (at >= 0) & (at < (s["start"][1:] - s["start"][:-1]).long()[of][:, None])
    if c["mask"] == "causal":
        drafted &= at <= s["node"][:, None]
    if s["mask"] is not None:
        n = at.clamp(min=0, max=64 * s["mask"].shape[1] - 1)
        drafted &= (s["mask"].gather(1, n // 64) >> (n % 64)) & 1 == 1
    seen = torch.zeros((B, Q, j.numel()), dtype=torch.bool, device="cuda")
    seen[of, s["node"]] = (at < 0) | drafted
    x.view(B, H // G, Q, G, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _plain_rows(s, 1).permute(0, 2, 1, 3)) / torch.where(total == 0, torch.ones_like(total), total)
    back = lambda y: y.reshape(B, H // G, Q, G, -1).permute(0, 2, 1, 3, 4).reshape(B, Q, H, -1)[of, s["node"]]  # noqa: E731
    return {"out": back(o).to(torch.bfloat16), "lse": back(total.log() + top)[..., 0]}


# ------------------------------------------------------------------ one pass


def run(state):
    s = state
    if not own:
        return {"verify": _plain_verify, "compact": _plain_compact, "pages": _plain_pages, "insert": _plain_insert, "attention": _plain_attention}[s["op"]](s)
    import speculative_decoding_draft_ctx_gb300 as dk

    c = s["c"]
    if s["op"] == "verify":
        tokens, rows, counts = dk.verify_drafts(s["target"], s["tokens"], s["start"], s["uniforms"], _depth(c), draft_probs=s["draft"], parents=s["parents"],
                                                replacement=c["replacement"])
        return {"tokens": tokens, "rows": rows, "counts": counts}
    if s["op"] == "compact":
        lens = dk.compact_kv(s["caches"], s["table"], s["ctx"], s["rows"], s["counts"], block_scales=s["scales"])
        out = {"lens": lens, "caches": [_view(s, x) for x in s["caches"]]}
        if s["scales"] is not None:
            out["scales"] = s["scales"]
        return out
    if s["op"] == "pages":
        _restore(s)
        dk.fork_kv(s["caches"], s["table"], s["pages"], s["lens"], s["src"], s["dst"], s["refs"], block_scales=s["scales"])
        lens = s["lens"]
        want = torch.where(s["keep"] & (lens > 0), lens + c["draft"], 0)
        dk.resize_kv(s["table"], s["pages"], want, s["refs"], c["block"])
        return _pages_out(s)
    if s["op"] == "insert":
        dk.insert_kv_scaled(s["k"], s["v"], s["cache"], s["scales"], s["table"], s["start"], s["ctx"])
        return {"cache": s["cache"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    out, lse = dk.tree_attention(s["q"], s["cache"], s["table"], s["start"], s["ctx"], tree_mask=s["mask"], causal=c["mask"] == "causal",
                                 block_scales=s["scales"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ floors


def work(case):
    c = case
    if c["op"] == "verify":
        size, n, B, V = 2 if c["bf16"] else 4, sum(_drafts(c)), c["requests"], c["vocab"]
        # a request's draw reads one row of each, its tests one entry of each
        each = 2 if c["draft"] == "probs" else 1
        return {"bytes": B * V * each * size + n * (each * size + 16) + B * (_depth(c) * 12 + 20), "flops": 3 * B * V}
    row = 2 * c["dim"] * c["kv_heads"] * (2 if c.get("kind") == "bf16" else 1)  # a token's K|V in a layer
    if c["op"] == "compact":
        most = sum(min(c["accept"], n // 2) for n in _drafts(c))
        return {"bytes": most // 4 * 2 * row * c["layers"] + c["requests"] * (c["accept"] * 4 + 12), "flops": 0}
    if c["op"] == "pages":
        lens = _spread(c["live"], c["ctx_min"], c["ctx_max"], 0.618034)[c["finished"]:]
        tails = [lens[i % min(16, len(lens))] % c["block"] for i in range(c["forks"])]
        entries = sum(lens[i % min(16, len(lens))] // c["block"] for i in range(c["forks"]))
        return {"bytes": sum(tails) * 2 * row * c["layers"] + entries * 16 + c["pool"] * 4, "flops": 0}
    ctx, q = _lengths(c)
    T, H, D = sum(q), c["kv_heads"], c["dim"]
    if c["op"] == "insert":
        return {"bytes": T * H * 2 * D * 3 + T * 8, "flops": 4 * T * H * D}
    total = sum(n + m for n, m in zip(ctx, q))
    return {"bytes": total * H * 2 * D + sum(-(-(n + m) // c["block"]) for n, m in zip(ctx, q)) * (2 * H + 4) + T * c["heads"] * (4 * D + 4),
            "flops": sum(4 * D * m * c["heads"] * (n + m) for n, m in zip(ctx, q))}


# ------------------------------------------------------------------ from the definitions, in 64 bits


def _exact_verify(s):
    import numpy as np

    c, depth = s["c"], _depth(s["c"])
    start, tokens, u = s["start"].tolist(), s["tokens"].tolist(), s["uniforms"].double().tolist()
    B = len(start) - 1
    out_t, out_r, out_n = np.full((B, depth + 1), -1, np.int64), np.full((B, depth), -1, np.int32), np.zeros(B, np.int32)
    numbers = lambda x, t: x[t].double().cpu().numpy()  # noqa: E731
    for b in range(B):
        lo, n = start[b], start[b + 1] - start[b]
        up = [-1] + (list(range(n - 1)) if s["parents"] is None else s["parents"][lo + 1:lo + n].tolist())
        at = 0
        while True:
            p = numbers(s["target"], lo + at)
            q = None if s["draft"] is None else numbers(s["draft"], lo + at)
            rest, base = p.copy(), 1.0  # what is left of p; the mass that it stands for
            without = 0.0 if q is None else q.copy()
            step = None
            if out_n[b] < depth:
                for i in range(1, n):
                    if up[i] != at:
                        continue
                    x, v = tokens[lo + i], u[lo + i]
                    if q is None:
                        if base <= 0:
                            break
                        if v * base < rest[x]:
                            step = i
                            break
                        base -= rest[x]
                        rest[x] = 0.0
                        continue
                    left = 1.0 - (q.sum() - without.sum()) if not c["replacement"] else 1.0
                    if left <= 2.0 ** -24 or base <= 0:
                        break
                    if v * (q[x] / left) * base < rest[x]:
                        step = i
                        break
                    rest = np.maximum(rest - base * (without / left), 0.0)
                    rest[x] = 0.0
                    if not c["replacement"]:
                        without[x] = 0.0
                    base = rest.sum()
            if step is None:
                break
            out_t[b, out_n[b]], out_r[b, out_n[b]] = tokens[lo + step], step
            out_n[b] += 1
            at = step
        if not rest.sum() > 0:
            rest = p
        cum = np.cumsum(rest)
        out_t[b, out_n[b]] = min(int(np.searchsorted(cum, u[lo] * cum[-1], side="right")), int(np.flatnonzero(rest)[-1]))
    return {"tokens": torch.from_numpy(out_t), "rows": torch.from_numpy(out_r), "counts": torch.from_numpy(out_n)}


def _value(codes, e, D):
    """Codes [H, n, 2 D] with exponents [H, 2], as numbers in 64 bits."""
    x = codes.view(torch.float8_e4m3fn).double()
    return torch.cat([torch.ldexp(x[..., :D], e[:, None, :1].double()), torch.ldexp(x[..., D:], e[:, None, 1:].double())], -1)


def _encode(x, e, D):
    y = torch.cat([torch.ldexp(x[..., :D], -e[:, None, :1].double()), torch.ldexp(x[..., D:], -e[:, None, 1:].double())], -1)
    return y.clamp(-FP8_MAX, FP8_MAX).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)


def _exact_compact(s):
    c, bs, D = s["c"], s["c"]["block"], s["c"]["dim"]
    table, rows, counts, ctx = s["table"].tolist(), s["rows"].tolist(), s["counts"].tolist(), s["ctx"].tolist()
    for layer, cache in enumerate(s["caches"]):
        before = cache.clone()
        for b in range(len(ctx)):
            moves = [(ctx[b] + rows[b][j], ctx[b] + 1 + j) for j in range(counts[b]) if rows[b][j] != j + 1]
            if s["scales"] is None:
                for of, to in moves:
                    cache[table[b][to // bs], :, to % bs] = before[table[b][of // bs], :, of % bs]
                continue
            sc = s["scales"][layer]
            was = {p: sc[p].clone() for p in {table[b][x // bs] for m in moves for x in m}}
            for k in sorted({to // bs for _, to in moves}):
                page = table[b][k]
                into = [m for m in moves if m[1] // bs == k]
                e = torch.stack([was[page]] + [was[table[b][of // bs]] for of, _ in into]).amax(0)
                kept = _encode(_value(before[page], was[page], D), e, D)
                same = (e == was[page]).repeat_interleave(D, -1)[:, None]
                cache[page] = torch.where(same, before[page], kept)
                for of, to in into:
                    x = _value(before[table[b][of // bs], :, of % bs][:, None], was[table[b][of // bs]], D)
                    cache[page, :, to % bs] = _encode(x, e, D)[:, 0]
                sc[page] = e
    out = {"lens": torch.tensor([n + 1 + k for n, k in zip(ctx, counts)], dtype=torch.int32), "caches": [_view(s, x) for x in s["caches"]]}
    if s["scales"] is not None:
        out["scales"] = s["scales"]
    return out


def _exact_pages(s):
    import heapq

    c, bs = s["c"], s["c"]["block"]
    table, refs, pages, lens = (s["held"][k].tolist() for k in ("table", "refs", "pages", "lens"))
    free = [p for p, n in enumerate(refs) if n == 0]
    heapq.heapify(free)
    for a, d in zip(s["src"].tolist(), s["dst"].tolist()):
        full, tail = divmod(lens[a], bs)
        for k in range(full):
            table[d][k] = table[a][k]
            refs[table[a][k]] += 1
        if tail:
            page, old = heapq.heappop(free), table[a][full]
            refs[page] = 1
            table[d][full] = page
            for layer, cache in enumerate(s["caches"]):
                cache[page, :, :tail] = cache[old, :, :tail]
                if s["scales"] is not None:
                    s["scales"][layer][page] = s["scales"][layer][old]
        pages[d], lens[d] = full + (tail > 0), lens[a]
    keep = s["keep"].tolist()
    need = [-(-(n + c["draft"]) // bs) if k and n else 0 for n, k in zip(lens, keep)]
    for r in range(len(need)):
        while pages[r] > need[r]:
            pages[r] -= 1
            page = table[r][pages[r]]
            table[r][pages[r]] = -1
            refs[page] -= 1
            if refs[page] == 0:
                heapq.heappush(free, page)
    for r in range(len(need)):
        while pages[r] < need[r]:
            page = heapq.heappop(free)
            refs[page] = 1
            table[r][pages[r]] = page
            pages[r] += 1
    as_int = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    out = {"table": as_int(table), "refs": as_int(refs), "pages": as_int(pages), "lens": as_int(lens), "caches": [_view(s, x) for x in s["caches"]]}
    if s["scales"] is not None:
        out["scales"] = s["scales"]
    return out


def _exact_insert(s):
    c, bs, D = s["c"], s["c"]["block"], s["c"]["dim"]
    start, ctx, table = s["start"].tolist(), s["ctx"].tolist(), s["table"].tolist()
    for b in range(len(ctx)):
        x = torch.cat([s["k"][start[b]:start[b + 1]], s["v"][start[b]:start[b + 1]]], -1).double().transpose(0, 1)  # [H, n, 2 D]
        n, at = x.shape[1], 0
        while at < n:
            page, off = table[b][(ctx[b] + at) // bs], (ctx[b] + at) % bs
            m = min(bs - off, n - at)
            part = x[:, at:at + m]
            top = torch.stack([part[..., :D].abs().amax((1, 2)), part[..., D:].abs().amax((1, 2))], 1)
            sizes = FP8_MAX * 2.0 ** torch.arange(EXP_MIN, EXP_MAX, device="cuda", dtype=torch.float64)
            e = (sizes < top[..., None]).sum(-1).double() + EXP_MIN  # the first that holds the largest value
            was = s["scales"][page].double()
            if off:
                e = torch.maximum(e, was)
                kept = _encode(_value(s["cache"][page, :, :off], was, D), e, D)
                same = (e == was).repeat_interleave(D, -1)[:, None]
                s["cache"][page, :, :off] = torch.where(same, s["cache"][page, :, :off], kept)
            s["cache"][page, :, off:off + m] = _encode(part, e, D)
            s["scales"][page] = e.to(torch.int8)
            at += m
    return {"cache": s["cache"].view(torch.float8_e4m3fn), "scales": s["scales"]}


def _exact_attention(s):
    c, D = s["c"], s["c"]["dim"]
    G, bs = c["heads"] // c["kv_heads"], c["block"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    start, ctx = s["start"].tolist(), s["ctx"].tolist()
    for b, n in enumerate(ctx):
        lo, hi = start[b], start[b + 1]
        Q = hi - lo
        j = torch.arange(n + Q, device="cuda")
        page = s["table"][b].long()[j // bs]
        tail = torch.ones((Q, Q), dtype=torch.bool, device="cuda")
        if c["mask"] == "causal":
            tail = tail.tril()
        if s["mask"] is not None:
            tail = torch.stack([(s["mask"][lo:hi, i // 64] >> (i % 64)) & 1 for i in range(Q)], 1).bool()
        seen = torch.cat([torch.ones((Q, n), dtype=torch.bool, device="cuda"), tail], 1)[:, None]
        for h in range(c["kv_heads"]):
            x = s["cache"][page, h, j % bs].view(torch.float8_e4m3fn).double()
            e = s["scales"][page, h].double()
            k, v = torch.ldexp(x[:, :D], e[:, :1]), torch.ldexp(x[:, D:], e[:, 1:])
            scores = ((s["q"][lo:hi, h * G:(h + 1) * G].double() @ k.T) * D ** -0.5).masked_fill(~seen, -math.inf)
            z = torch.logsumexp(scores, -1)
            out[lo:hi, h * G:(h + 1) * G] = (scores - z[..., None]).exp() @ v
            lse[lo:hi, h * G:(h + 1) * G] = z
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"verify": _exact_verify, "compact": _exact_compact, "pages": _exact_pages, "insert": _exact_insert, "attention": _exact_attention}[s["op"]](s)
