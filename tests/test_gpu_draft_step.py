"""The draft-step operators against their plain 64-bit forms (GB300)."""

import math
import random

import pytest
import torch

import speculative_decoding_draft_ctx_gb300 as dk
from draft_attn_ref import attention, close, gen, tree_mask
from draft_step_ref import EXP_MAX, EXP_MIN, Pool, ScaledProblem, compact, encode, insert_scaled, value, verify

pytestmark = pytest.mark.gpu


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ verification


def probabilities(rows, V, g, sharp=3.0, dtype=torch.float32):
    return torch.softmax(torch.randn((rows, V), generator=g) * sharp, 1).to(dtype)


def draws(V, drafts, g, arity=1, distinct=False, target_dtype=torch.float32, draft_dtype=torch.float32):
    """A batch: distributions near one another, tokens drawn from the drafter's, parents of trees."""
    r = random.Random(V)
    start = [0]
    for n in drafts:
        start.append(start[-1] + (n + 1 if n >= 0 else 0))
    T = start[-1]
    logits = torch.randn((T, V), generator=g) * 3
    target = torch.softmax(logits, 1).to(target_dtype)
    draft = torch.softmax(logits + torch.randn((T, V), generator=g), 1).to(draft_dtype)
    parents, tokens = torch.zeros(T, dtype=torch.int32), torch.zeros(T, dtype=torch.int64)
    for b, n in enumerate(drafts):
        seen = {}
        for i in range(1, n + 1):
            p = i - 1 if arity == 1 else r.choice([x for x in range(i) if len(seen.get(x, [])) < arity])
            q = draft[start[b] + p].double().clone()
            if distinct:
                q[seen.get(p, [])] = 0
            x = int(torch.multinomial(q, 1, generator=g)) if q.sum() > 0 else 0
            seen.setdefault(p, []).append(x)
            parents[start[b] + i], tokens[start[b] + i] = p, x
    return target, draft, tokens, torch.tensor(start, dtype=torch.int32), parents, torch.rand(T, generator=g)


def check_verify(target, draft, tokens, start, parents, u, most, replacement=True, flags=0, place=lambda x: x.cuda()):
    f = flag()
    got = dk.verify_drafts(place(target), tokens.cuda(), start.cuda(), u.cuda(), most, draft_probs=None if draft is None else place(draft),
                           parents=None if parents is None else parents.cuda(), replacement=replacement, error_flags=f)
    want = verify(target, draft, tokens, start, parents, u, most, replacement)
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), y)
    assert int(f) == flags
    return got


VOCABS = [1, 2, 5, 127, 128, 129, 1000, 4097, 33000]


@pytest.mark.parametrize("dtypes", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                                    (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("V", VOCABS)
def test_verify_chains(V, dtypes):
    g = gen(V)
    t, d, tok, start, _, u = draws(V, [7, 0, 3, -1, 1, 12, 7, 5], g, target_dtype=dtypes[0], draft_dtype=dtypes[1])
    check_verify(t, d, tok, start, None, u, 12)
    check_verify(t, d, tok, start, None, u, 3)  # fewer accepted tokens than drafted ones
    check_verify(t, None, tok, start, None, u, 12)


@pytest.mark.parametrize("replacement", [True, False])
@pytest.mark.parametrize("V", VOCABS)
def test_verify_trees(V, replacement):
    g = gen(V + 1)
    arity = min(4, V)
    t, d, tok, start, up, u = draws(V, [20, 0, 63, -1, 9, 40], g, arity=arity, distinct=not replacement)
    check_verify(t, d, tok, start, up, u, 8, replacement)
    check_verify(t, d, tok, start, up, u * 0.9 + 0.1, 63, replacement)
    check_verify(t, None, tok, start, up, u, 8, replacement)


def test_verify_largest_request_and_a_row_more():
    g = gen(5)
    t, d, tok, start, up, u = draws(40, [1023, 2], g, arity=3)
    check_verify(t, d, tok, start, up, u, 1023)
    check_verify(t, d, tok, start, None, u, 1023)
    t, d, tok, start, up, u = draws(40, [1024, 2], g, arity=3)
    got = dk.verify_drafts(t.cuda(), tok.cuda(), start.cuda(), u.cuda(), 5, d.cuda(), up.cuda(), error_flags=(f := flag()))
    assert int(f) == dk.FLAG_LENGTH and int(got[2][0]) == 0 and bool((got[0][0] == -1).all())
    want = verify(t[1025:], d[1025:], tok[1025:], torch.tensor([0, 3]), up[1025:], u[1025:], 5, True)
    assert torch.equal(got[0][1].cpu(), want[0][0])


@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 5), (4, 4)])
def test_verify_rows_of_any_stride_and_alignment(offset, pad):
    g = gen(9)
    t, d, tok, start, up, u = draws(1001, [5, 9, 2], g, arity=2)

    def place(x):
        wide = torch.full((x.shape[0], offset + x.shape[1] + pad), float("nan"), dtype=x.dtype, device="cuda")
        wide[:, offset:offset + x.shape[1]] = x.cuda()
        return wide[:, offset:offset + x.shape[1]]

    check_verify(t, d, tok, start, up, u, 9, place=place)
    check_verify(t.bfloat16(), d.bfloat16(), tok, start, up, u, 9, place=place)


def test_verify_draws_over_a_large_vocabulary():
    """One token of 131,072: borders between tokens lie 2^-17 apart on average."""
    g = gen(2)
    V, B = 131072, 96
    t, d = probabilities(2, V, g, 2.0), probabilities(2, V, g, 2.0)
    rows = torch.arange(2 * B) % 2
    tok, start = torch.randint(0, V, (2 * B,), generator=g), torch.arange(0, 2 * B + 1, 2, dtype=torch.int32)
    u = torch.rand(2 * B, generator=g)
    check_verify(t[rows], d[rows], tok, start, None, u, 1)
    check_verify(t[rows], None, tok, start, None, u, 1)


def test_verify_gives_the_target_s_own_distribution():
    """Over a grid of random numbers, first tokens come as often as the target has them, however the drafts were drawn."""
    p, q = torch.tensor([0.5, 0.25, 0.125, 0.125]), torch.tensor([0.25, 0.125, 0.5, 0.125])
    n = 64
    mid = (torch.arange(n) + 0.5) / n
    for arity in (1, 2):
        grid = torch.cartesian_prod(mid[::8], mid, mid[::4], mid[::4]) if arity == 2 else torch.cartesian_prod(mid, mid)
        total = torch.zeros(4, dtype=torch.float64)
        for x in range(4):
            for y in range(4 if arity == 2 else 1):
                B, k = grid.shape[0], arity + 1
                tok = torch.zeros((B, k), dtype=torch.int64)
                tok[:, 1] = x
                u = torch.zeros((B, k))
                if arity == 2:
                    tok[:, 2] = y
                    u[:, 0], u[:, 1], u[:, 2] = grid[:, 1], grid[:, 2], grid[:, 3]
                    u[:, 0] = (u[:, 0] + grid[:, 0] / 64) % 1
                else:
                    u[:, 0], u[:, 1] = grid[:, 0], grid[:, 1]
                up = torch.zeros(B * k, dtype=torch.int32)
                tokens, _, _ = dk.verify_drafts(p.expand(B * k, 4).contiguous().cuda(), tok.flatten().cuda(),
                                                torch.arange(0, B * k + 1, k, dtype=torch.int32).cuda(), u.flatten().cuda(), 1,
                                                q.expand(B * k, 4).contiguous().cuda(), up.cuda() if arity == 2 else None)
                share = torch.bincount(tokens[:, 0].cpu(), minlength=4).double() / B
                total += share * float(q[x]) * (float(q[y]) if arity == 2 else 1.0)
        # each border of a test or draw is met to a grid step: at most two steps of each random number
        assert (total - p.double()).abs().max() <= (2 / 16 if arity == 2 else 2 / 64), total


def test_verify_certain_rows():
    V = 300
    one = torch.zeros((4, V))
    one[:, 7] = 1.0
    tok, start, u = torch.tensor([0, 7, 7, 9]), torch.tensor([0, 4], dtype=torch.int32), torch.tensor([0.9999, 0.9999999, 0.5, 0.0])
    got = check_verify(one, one, tok, start, None, u, 3)  # p = q: accepted whatever u; 9 has neither
    assert got[0].tolist() == [[7, 7, 7, -1]] and got[1].tolist() == [[1, 2, -1]] and got[2].tolist() == [2]
    got = check_verify(one, None, tok, start, None, u, 3)
    assert got[0].tolist() == [[7, 7, 7, -1]]


def test_verify_where_the_rejections_leave_nothing():
    """p below q everywhere: the last token comes from p itself, and children that come up then are rejected."""
    V = 200
    q = torch.full((4, V), 1.0 / V)
    p = q * 0.5
    tok, start = torch.tensor([0, 3, 4, 5]), torch.tensor([0, 4], dtype=torch.int32)
    up = torch.zeros(4, dtype=torch.int32)
    got = check_verify(p, q, tok, start, up, torch.tensor([0.5, 0.75, 0.0, 0.0]), 3)
    assert got[2].tolist() == [0] and got[0][0, 0] == 100
    check_verify(p, q, tok, start, None, torch.tensor([0.25, 0.75, 0.0, 0.0]), 3)
    # the drafts without drawing cover all of p
    p = torch.zeros((3, V))
    p[:, 3] = 1.0
    got = check_verify(p, None, torch.tensor([0, 3, 3]), torch.tensor([0, 3], dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                       torch.tensor([0.2, float("nan"), 0.3]), 2)
    assert got[0][0, 0] == 3  # u that is not a number counts as 0


@pytest.mark.parametrize("draft", [True, False])
def test_verify_entries_and_numbers_out_of_range(draft):
    g = gen(4)
    t, d, tok, start, up, u = draws(500, [4, 4, 4], g, arity=2)
    t[0, :50], t[1, 3], t[2, 9], d[0, 5], d[5, 7] = float("nan"), -1.0, float("inf"), float("nan"), -2.0
    u[0], u[5], u[10], u[1] = 1.0, float("nan"), -3.0, 2.0
    check_verify(t, d if draft else None, tok, start, up, u, 4)
    tok[1], tok[7] = -1, 500
    check_verify(t, d if draft else None, tok, start, up, u, 4, flags=dk.FLAG_ROW)
    check_verify(t, d if draft else None, tok, start, None, u, 4, flags=dk.FLAG_ROW)
    tok[1], tok[7] = 3, 4
    up[2], up[8], up[13] = 2, -5, 70  # not rows before theirs
    check_verify(t, d if draft else None, tok, start, up, u, 4, flags=dk.FLAG_ROW)


def test_verify_a_row_without_any_probability():
    t = torch.zeros((3, 70))
    got = check_verify(t, None, torch.tensor([0, 1, 2]), torch.tensor([0, 3], dtype=torch.int32), None, torch.full((3,), 0.5), 2, flags=dk.FLAG_ROW)
    assert got[0].tolist() == [[-1, -1, -1]]


def test_verify_bad_rows_of_a_request():
    g = gen(6)
    t, d, tok, start, _, u = draws(100, [3, 3, 3], g)
    for bad in ([0, 13, 8, 12], [-1, 4, 8, 12], [0, 4, 8, 13]):
        f = flag()
        out = dk.verify_drafts(t.cuda(), tok.cuda(), ints(bad), u.cuda(), 3, d.cuda(), error_flags=f)
        assert int(f) == dk.FLAG_LENGTH
        want = verify(t, d, tok, start, None, u, 3, True)
        for b in range(3):
            if bad[b] == int(start[b]) and bad[b + 1] == int(start[b + 1]):
                assert torch.equal(out[0][b].cpu(), want[0][b])


def test_verify_in_a_graph_and_on_another_stream():
    g = gen(8)
    t, d, tok, start, up, u = draws(5000, [9, 20, 5], g, arity=3)
    args = [x.cuda() for x in (t, tok, start, u)]
    d, up = d.cuda(), up.cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out = dk.verify_drafts(*args, 8, d, up, stream=stream)
    stream.synchronize()
    want = verify(t, d.cpu(), tok, start, up.cpu(), u, 8, True)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dk.verify_drafts(*args, 8, d, up)
    for k in range(3):
        u = torch.rand(u.shape, generator=g)
        args[3].copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        want = verify(t, d.cpu(), tok, start, up.cpu(), u, 8, True)
        assert all(torch.equal(a.cpu(), b) for a, b in zip(out, want))


# ------------------------------------------------------------------ compaction


def caches_of(kind, layers, blocks, H, bs, D, g):
    """Random layers' caches (every byte pattern of codes and of bf16 numbers) and their exponents."""
    if kind == "bf16":
        return [torch.randn((blocks, H, bs, 2 * D), generator=g).bfloat16() for _ in range(layers)], None
    caches = [torch.randint(0, 256, (blocks, H, bs, 2 * D), generator=g).to(torch.uint8) for _ in range(layers)]
    return caches, [torch.randint(-9, 9, (blocks, H, 2), generator=g).to(torch.int8) for _ in range(layers)] if kind == "scaled" else None


def same_codes(got, want):
    """Equal bytes, but for the sign of a zero or NaN."""
    if got.dtype is torch.uint8:
        a, b = got.cpu(), want
        zero = ((a & 0x7f) == 0) & ((b & 0x7f) == 0)
        nan = ((a & 0x7f) == 0x7f) & ((b & 0x7f) == 0x7f)
        return bool(((a == b) | zero | nan).all())
    return torch.equal(got.cpu(), want)


def check_compact(kind, ctx, paths, H, D, bs, layers=2, first=1, width=None, cols=None, edit=None, flags=0, seed=0, counts=None, most_pages=None):
    g = gen(seed + bs + D)
    B = len(ctx)
    width = width or max(1, max(len(p) for p in paths))
    need = [min(-(-(max(0, c) + max([0] + p) + 1) // bs), most_pages or 1 << 30) for c, p in zip(ctx, paths)]
    cols = cols or max(need)
    blocks = sum(need) + 2
    order, at = torch.randperm(blocks, generator=g), 0
    table = torch.full((B, cols), -7, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n][:cols].to(torch.int32)
        at += n
    caches, scales = caches_of(kind, layers, blocks, H, bs, D, g)
    rows = torch.full((B, width), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        rows[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    counts = [len(p) for p in paths] if counts is None else counts
    if edit:
        edit(table)
    d = [x.cuda() for x in caches]
    s = None if scales is None else [x.cuda() for x in scales]
    f = flag()
    lens = dk.compact_kv(d, table.cuda(), ints(ctx), rows.cuda(), ints(counts), first, block_scales=s, error_flags=f)
    want, ws, wl = compact(caches, scales, table, ctx, rows, counts, first, bs)
    assert lens.tolist() == wl
    for x, y in zip(d, want):
        assert same_codes(x, y)
    if s is not None:
        for x, y in zip(s, ws):
            assert torch.equal(x.cpu(), y)
    assert int(f) == flags
    return lens


PATHS = [[2, 3, 4], [1, 2, 3], [], [1, 3, 4, 7, 8, 20], [5], [40, 41, 42], [2, 4, 6, 8, 10, 12, 14, 16, 18, 20, 22, 24]]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "scaled"])
@pytest.mark.parametrize("bs,D,H", [(1, 64, 3), (3, 128, 2), (16, 128, 8), (16, 64, 1), (100, 256, 5), (64, 256, 3)])
def test_compact(kind, bs, D, H):
    """Paths that overlap the rows they move into, stay, leave at once or are empty."""
    check_compact(kind, [0, 5, 9, 14, 15, 16, 200], PATHS, H, D, bs)


@pytest.mark.parametrize("kind", ["bf16", "scaled"])
@pytest.mark.parametrize("bs", [5, 400])
def test_compact_long_paths(kind, bs):
    """More moves than are looked up at once, into many pages and into one."""
    check_compact(kind, [3, 70], [list(range(2, 1202, 2)), list(range(300, 900))], 1, 64, bs, layers=1)


@pytest.mark.parametrize("kind", ["bf16", "scaled"])
def test_compact_many_layers_and_first(kind):
    check_compact(kind, [7, 8], [[1, 2, 5], [0, 3]], 2, 64, 4, layers=70, first=0)
    check_compact(kind, [7, 8], [[5, 9], [6]], 2, 64, 4, layers=1, first=5)


@pytest.mark.parametrize("kind", ["bf16", "scaled"])
def test_compact_leaves_out_what_is_out_of_range(kind):
    for path, count, ctx in (([3, 2], None, 4), ([2, 2], None, 4), ([0, 3], None, 4), ([1, 3], 3, 4), ([1, 3], -1, 4), ([1, 3], None, -2)):
        check_compact(kind, [6, ctx], [[2, 4], path], 2, 64, 8, counts=None if count is None else [2, count], flags=dk.FLAG_LENGTH)
    check_compact(kind, [6, 3], [[2, 4], [1, 2 ** 31 - 2]], 2, 64, 8, cols=3, flags=dk.FLAG_LENGTH, most_pages=3)
    # behind the table's last entry
    check_compact(kind, [6, 20], [[2, 4], [2, 9]], 2, 64, 8, cols=3, flags=dk.FLAG_LENGTH)
    # a page out of range: its rows stay
    check_compact(kind, [6, 20], [[2, 4, 9], [2, 9]], 2, 64, 4, edit=lambda t: t.__setitem__((0, 2), 10 ** 6), flags=dk.FLAG_BLOCK_RANGE)
    check_compact(kind, [6, 20], [[2, 4, 9], [2, 9]], 2, 64, 4, edit=lambda t: t.__setitem__((0, 1), -1), flags=dk.FLAG_BLOCK_RANGE)


def test_compact_scales_far_apart():
    """Exponents 63 apart: codes become zero or stay, NaN stays."""
    g = gen(1)
    cache = torch.randint(0, 256, (3, 1, 4, 128), generator=g).to(torch.uint8)
    scales = torch.tensor([[[-32, 31]], [[31, -32]], [[127, -128]]], dtype=torch.int8)  # the last: taken as 31 and -32
    table, rows = torch.tensor([[0, 1, 2]], dtype=torch.int32), torch.tensor([[5, 10]], dtype=torch.int32)
    want, ws, _ = compact([cache], [scales.clamp(EXP_MIN, EXP_MAX)], table, [0], rows, [2], 1, 4)
    c, s = cache.cuda(), scales.cuda()
    dk.compact_kv(c, table.cuda(), ints([0]), rows.cuda(), ints([2]), block_scales=s)
    assert same_codes(c, want[0]) and s.cpu()[:2].tolist() == ws[0][:2].tolist()


# ------------------------------------------------------------------ the pool


class Live:
    """A Pool of the reference beside the device's tensors."""

    def __init__(self, rows, width, pages, bs, kind="bf16", layers=2, H=2, D=64, seed=0, wide=0):
        self.ref, self.bs = Pool(rows, width, pages, bs), bs
        g = gen(seed)
        self.caches, self.scales = caches_of(kind, layers, pages, H, bs, D, g)
        self.d_caches, self.d_scales = [x.cuda() for x in self.caches], None if self.scales is None else [x.cuda() for x in self.scales]
        self.full = torch.full((rows, width + wide), -1, dtype=torch.int32, device="cuda")
        self.table = self.full[:, :width]
        self.pages, self.lens, self.refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (rows, rows, pages))
        self.flags = flag()

    def resize(self, tokens):
        self.ref.resize(tokens)
        dk.resize_kv(self.table, self.pages, ints(tokens), self.refs, self.bs, error_flags=self.flags)

    def set_lens(self, lens):
        self.ref.lens = list(lens)
        self.lens.copy_(ints(lens))

    def fork(self, pairs):
        self.ref.copies.clear()
        self.ref.fork(pairs)
        for old, new, n in self.ref.copies:
            for layer, c in enumerate(self.caches):
                c[new, :, :n] = c[old, :, :n]
                if self.scales is not None:
                    self.scales[layer][new] = self.scales[layer][old]
        dk.fork_kv(self.d_caches, self.table, self.pages, self.lens, ints([p[0] for p in pairs]), ints([p[1] for p in pairs]), self.refs,
                   block_scales=self.d_scales, error_flags=self.flags)

    def check(self, flags=0):
        assert self.table.tolist() == self.ref.table
        assert self.pages.tolist() == self.ref.pages and self.lens.tolist() == self.ref.lens and self.refs.tolist() == self.ref.refs
        for a, b in zip(self.d_caches, self.caches):
            assert torch.equal(a.cpu(), b)
        for a, b in zip(self.d_scales or [], self.scales or []):
            assert torch.equal(a.cpu(), b)
        assert int(self.flags) == flags
        self.flags.zero_()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "scaled"])
@pytest.mark.parametrize("bs,D", [(16, 128), (1, 64), (5, 64), (48, 256)])
def test_pool_fork_and_resize(kind, bs, D):
    live = Live(9, 12, 70, bs, kind, D=D, wide=3)
    live.resize([3 * bs, 1, 0, 2 * bs + 1, bs, 0, 0, 0, 0])
    live.check()
    live.set_lens([3 * bs, 1, 0, 2 * bs, bs - 1, 0, 0, 0, 0])
    live.fork([(0, 5), (1, 2), (3, 6), (4, 7), (4, 8)])  # full pages alone, a part, pages held beyond the tokens, one twice
    live.check()
    live.resize([0, 4 * bs, bs, 12 * bs, 0, 3 * bs, 2 * bs, bs, 1])  # shared pages given back stay held by their others
    live.check()
    live.resize([0] * 9)
    assert live.ref.refs == [0] * 70
    live.check()


def test_pool_random_steps():
    """Forks, growth, shrinking and frees in turn: the pool's counts stay what the tables hold."""
    r = random.Random(3)
    live = Live(40, 30, 600, 8, "scaled", layers=1)
    for step in range(25):
        lens = [min(p * 8, max(0, n + r.randint(-9, 9))) for p, n in zip(live.ref.pages, live.ref.lens)]
        live.set_lens(lens)
        free = [i for i in range(40) if live.ref.pages[i] == 0]
        held = [i for i in range(40) if live.ref.pages[i]]
        if free and held:
            live.set_lens([0 if i in free else n for i, n in enumerate(live.ref.lens)])
            k = r.randint(1, len(free))
            live.fork([(r.choice(held), d) for d in r.sample(free, k)])
        want = [0 if r.random() < 0.15 else n + r.randint(0, 40) for n in live.ref.lens]
        before = live.ref.refs.count(0)
        asked = sum(max(0, -(-w // 8) - p) for w, p in zip(want, live.ref.pages))
        if asked > before:
            want = [min(w, p * 8) for w, p in zip(want, live.ref.pages)]
        live.resize(want)
        live.set_lens([min(n, p * 8) for n, p in zip(live.ref.lens, live.ref.pages)])
        live.check()
        counts = [0] * 600
        for row, n in zip(live.ref.table, live.ref.pages):
            for p in row[:n]:
                counts[p] += 1
        assert counts == live.ref.refs


def test_pool_fork_of_many_pairs_and_long_rows():
    n = 300
    live = Live(n + 3, 400, 2000, 4, layers=1, H=1)
    live.resize([1597, 0 + 7, 400] + [0] * n)
    live.set_lens([1597, 7, 400] + [0] * n)
    live.fork([(i % 3, 3 + i) for i in range(n)])
    live.check()
    live.resize([0, 0, 0] + [1600 if i % 3 == 0 else 0 for i in range(n)])
    live.check()


def test_pool_runs_out():
    live = Live(6, 8, 10, 4, layers=1)
    live.resize([12, 5, 9, 4, 1, 0])  # 3 + 2 + 3 + 1 + 1 of 10
    live.check()
    live.set_lens([10, 5, 9, 4, 1, 0])
    live.fork([(0, 5)])
    live.check(dk.FLAG_PAGES)
    live.resize([12, 20, 0, 9, 8, 4])  # 3 come free: row 1 asks for 3 and gets them, the others nothing
    live.check(dk.FLAG_PAGES)
    live.resize([0, 20, 0, 13, 1, 9])  # 3 free: row 3 asks for 3 and gets them, row 5 asks for 3 and does not
    live.check(dk.FLAG_PAGES)
    # the pairs in need get pages in their order
    live = Live(8, 2, 5, 4, layers=1)
    live.resize([3, 2, 4, 0, 0, 0, 0, 0])
    live.set_lens([3, 2, 4, 0, 0, 0, 0, 0])
    live.fork([(2, 7), (0, 3), (1, 4), (0, 5), (2, 6)])
    assert live.ref.pages == [1, 1, 1, 1, 1, 0, 1, 1]
    live.check(dk.FLAG_PAGES)


def test_pool_fork_leaves_out_unsound_pairs():
    live = Live(8, 4, 40, 4, layers=1)
    live.resize([9, 6, 3, 0, 0, 0, 0, 0])
    live.set_lens([9, 6, 3, 0, 0, 0, 0, 0])
    live.fork([(0, 1), (0, 3), (1, 3), (3, 4), (-1, 5), (8, 5), (0, 8), (1, 6), (2, 2)])  # held; 3 is a src; twice; ranges; itself
    live.check(dk.FLAG_LENGTH)
    assert live.ref.pages == [3, 2, 1, 0, 0, 0, 2, 0]
    live.set_lens([13, 6, -1, 0, 0, 0, 6, 0])  # more tokens than pages, fewer than none
    live.fork([(0, 4), (2, 5), (1, 7)])
    live.check(dk.FLAG_LENGTH)
    # entries out of range: the last page's leaves the pair out, others are copied as they are
    for row, at in ((1, 1), (0, 1)):
        live.table[row, at] = 99
        live.ref.table[row][at] = 99
    live.set_lens([9, 6, 3, 0, 0, 0, 6, 6])
    live.fork([(1, 3), (0, 4)])
    live.check(dk.FLAG_BLOCK_RANGE)


def test_pool_resize_of_bad_rows_and_entries():
    live = Live(5, 4, 20, 4, layers=1)
    live.resize([16, 8, 4, 0, 0])
    live.resize([17, 8, -1, 4, 0])  # beyond the table; fewer than none
    live.check(dk.FLAG_LENGTH)
    live.table[0, 3], live.table[1, 1] = 20, live.table[0, 0].clone()
    live.ref.table[0][3], live.ref.table[1][1] = 20, live.ref.table[0][0]
    live.resize([8, 0, 4, 4, 0])
    live.check(dk.FLAG_BLOCK_RANGE)
    live.resize([0, 0, 4, 4, 0])  # page 0 was given back by row 1 already: nobody held it
    live.check(dk.FLAG_REFS)


@pytest.mark.parametrize("offset,pages", [(1, 5000), (0, 8193), (3, 70001), (0, 200003)])
def test_pool_of_any_size_and_alignment(offset, pages):
    """Runs of a thread of several loads, pools that no thread's run divides, refs at any address."""
    live = Live(6, 40, 8, 4, layers=1, H=1)
    live.ref.refs = [int(x) for x in (torch.rand(pages, generator=gen(pages)) < 0.98)]
    full = torch.zeros(pages + offset, dtype=torch.int32, device="cuda")
    live.refs = full[offset:]
    live.refs.copy_(ints(live.ref.refs))
    # the caches play no part here: one of a page
    live.resize([160, 3, 0, 77, 4, 1])
    assert live.table.tolist() == live.ref.table and live.refs.tolist() == live.ref.refs
    live.resize([1, 3, 100, 160, 0, 9])
    assert live.table.tolist() == live.ref.table and live.refs.tolist() == live.ref.refs and live.pages.tolist() == live.ref.pages
    assert int(live.flags) == 0


def test_pool_resize_of_many_rows():
    """More rows than the cluster has threads, more pages than one round of them."""
    n = 9000
    live = Live(n, 3, 20000, 2, layers=1, H=1)
    live.resize([i % 5 for i in range(n)])
    live.check()
    live.resize([(i * 7) % 7 if i % 3 else 0 for i in range(n)])
    live.check()


# ------------------------------------------------------------------ page-scaled caches: the insert


def check_insert(ctx, nq, H, D, bs, seed=0, packed=False, edit=None, flags=0, spread=3.0, table_edit=None):
    g = gen(seed + D + bs)
    p = ScaledProblem(seed, ctx, nq, H, H, D, bs)
    T = sum(nq)
    x = torch.randn((T, 3 * H, D), generator=g) * torch.exp(torch.randn((T, 3 * H, 1), generator=g) * spread)
    x = x.bfloat16()
    if edit:
        edit(x)
    if table_edit:
        table_edit(p.table)
    k, v = (x[:, H:2 * H], x[:, 2 * H:]) if packed else (x[:, :H].contiguous(), x[:, H:2 * H].contiguous())
    want, ws = insert_scaled(k, v, p.cache, p.scales, p.table, p.start, p.ctx, bs)
    dx = x.cuda()
    dk_, dv = (dx[:, H:2 * H], dx[:, 2 * H:]) if packed else (k.cuda(), v.cuda())
    p.cuda()
    dk.insert_kv_scaled(dk_, dv, p.d_cache, p.d_scales, p.d_table, p.d_start, p.d_ctx, error_flags=p.d_flags)
    assert torch.equal(p.d_scales.cpu(), ws)
    assert same_codes(p.d_cache, want)
    assert int(p.d_flags) == flags
    return p


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [1, 3, 16, 64, 100, 300])
def test_insert_scaled(D, bs):
    check_insert((0, 5, 16, 31, 100, 0), (7, 1, 3, 0, 20, 130), 3, D, bs, packed=bs % 2 == 0)


def test_insert_scaled_single_tokens_of_many_requests():
    n = 700
    check_insert(tuple(i % 37 for i in range(n)), tuple(int(i % 5 != 0) for i in range(n)), 2, 64, 16)


def test_insert_scaled_values_at_the_ends():
    """Zeros, numbers below the least scale and above the largest, infinities, NaN, and exactly 448 times a power of two."""
    def edit(x):
        x[0] = 0.0
        x[1] = 2.0 ** -100
        x[2, :, 3] = float("inf")
        x[3, :, 4] = float("nan")
        x[4] = 3e38
        x[5] = 448 * 2.0 ** -7
        x[6] = 450 * 2.0 ** -7
        x[7] = float("-inf")
    for ctx in ((0,) * 8, (3,) * 8):
        check_insert(ctx, (1,) * 8, 2, 64, 4, edit=edit)


def test_insert_scaled_leaves_out_what_is_out_of_range():
    check_insert((4, 6, 9), (3, 4, 5), 2, 64, 4, table_edit=lambda t: t.__setitem__((1, 2), 10 ** 6), flags=dk.FLAG_BLOCK_RANGE)
    p = ScaledProblem(1, (4, 6, 9), (3, 4, 5), 2, 2, 64, 4).cuda()
    before, k = p.d_cache.clone(), torch.randn((12, 2, 64), device="cuda").bfloat16()
    for start, ctx in (([0, 3, 2, 12], (4, 6, 9)), ([0, 3, 7, 13], (4, 6, 9)), ([0, 3, 7, 12], (4, 6, 12)), ([0, 3, 7, 12], (4, 6, -1))):
        p.d_cache.copy_(before)
        p.d_flags.zero_()
        dk.insert_kv_scaled(k, k, p.d_cache, p.d_scales, p.d_table, ints(start), ints(ctx), error_flags=p.d_flags)
        assert int(p.d_flags) == dk.FLAG_LENGTH
        page = p.table[2].long()[:3]
        assert torch.equal(p.d_cache.cpu()[page], before.cpu()[page])


# ------------------------------------------------------------------ page-scaled caches: the attention


def run_scaled(p, kind, mask, **kw):
    return dk.tree_attention(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, tree_mask=mask.cuda() if kind == "tree" else None,
                             causal=kind == "causal", error_flags=p.d_flags, block_scales=p.d_scales, **kw)


def check_scaled(p, kind, mask, **kw):
    p.cuda()
    out, lse = run_scaled(p, kind, mask, **kw)
    want, z, to, tl = attention(p, kind, mask)
    close(lse, z, tl)
    close(out, want, to)
    assert int(p.d_flags) == 0
    return out, lse


SCALED = [
    ((300,), (1,), 8, 8, 128, 16, "dense"),
    ((300,), (7,), 64, 8, 128, 16, "dense"),
    ((0, 5, 63, 64, 65, 700), (1, 3, 7, 2, 5, 6), 6, 2, 64, 16, "causal"),
    ((0, 1, 200, 33), (9, 0, 1, 20), 10, 2, 128, 1, "tree"),
    ((130, 40), (64, 70), 8, 2, 128, 100, "tree"),
    ((1000, 3), (5, 5), 4, 4, 256, 48, "causal"),
    ((4000, 300), (64, 33), 32, 4, 64, 16, "tree"),
    ((3000, 0, 700), (64, 5, 20), 40, 8, 128, 64, "tree"),
    ((2500, 129), (30, 70), 20, 4, 256, 100, "causal"),
    ((12000,), (1,), 8, 1, 128, 128, "dense"),
    (tuple(range(0, 300)), tuple(i % 3 for i in range(300)), 2, 2, 64, 16, "causal"),
]


@pytest.fixture(params=["default", "mma", "tc"])
def kernel(request, monkeypatch):
    if request.param != "default":
        monkeypatch.setenv("DSPARK_TREE_ATTN_KERNEL", request.param)
    return request.param


@pytest.mark.parametrize("ctx,nq,Hq,Hkv,D,bs,kind", SCALED)
def test_scaled_attention(ctx, nq, Hq, Hkv, D, bs, kind, kernel):
    p = ScaledProblem(len(ctx) + D + bs, ctx, nq, Hq, Hkv, D, bs, packed=True)
    mask = tree_mask(nq, max(1, -(-max(nq) // 64)), D, empty=(0,) if sum(nq) else ())
    check_scaled(p, kind, mask)


@pytest.mark.parametrize("D,nq", [(64, 1), (128, 1), (128, 20), (256, 3)])
def test_scaled_attention_scales_far_apart(D, nq, kernel):
    """V's scales over their whole range, a heavy token in a page of small scale before light ones in pages of large scale."""
    p = ScaledProblem(3, (700, 64), (nq, nq), 8, 2, D, 16, v_exp=(-32, 32))
    check_scaled(p, "dense", None)
    p = ScaledProblem(4, (700, 64), (nq, nq), 8, 2, D, 16)
    for b in range(2):
        heavy = int(p.table[b, 1])
        p.scales[heavy, :, 1] = -32
        p.scales[heavy, :, 0] = 3   # scores of the heavy page beyond all others
        for k in range(2, 4):
            p.scales[int(p.table[b, k]), :, 1] = 31
    check_scaled(p, "dense", None)


def test_scaled_attention_is_the_plain_one_where_scales_are_alike(kernel):
    """One power of two for all pages: what the per-tensor scales give."""
    p = ScaledProblem(5, (500, 70), (9, 30), 16, 4, 128, 16, k_exp=(-5, -4), v_exp=(-6, -5)).cuda()
    a = run_scaled(p, "dense", None)
    b = dk.tree_attention(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, k_scale=torch.tensor([2.0 ** -5], device="cuda"),
                          v_scale=torch.tensor([2.0 ** -6], device="cuda"))
    assert (a[0].float() - b[0].float()).abs().max() <= 2.0 ** -7 * b[0].float().abs().max()
    assert (a[1] - b[1]).abs().max() <= 2.0 ** -18 * (1 + b[1].abs().max())


def test_scaled_attention_rows_without_anything_pages_and_lengths_out_of_range(kernel):
    p = ScaledProblem(3, (0, 40), (3, 2), 4, 2, 128, 16, pad_rows=3).cuda()
    mask = torch.tensor([[0], [2], [0], [0], [3], [-1], [-1], [-1]])
    out, lse = torch.full((8, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((8, 4), 7.0, device="cuda")
    run_scaled(p, "tree", mask, out=out, lse=lse)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all()) and bool((out[5:] == 7).all()) and bool((lse[5:] == 7).all())
    want, z, to, tl = attention(p, "tree", mask)
    close(out[:5], want, to)
    # a page out of range: its tokens are left out
    p.d_table[1, 1] = p.blocks
    out, lse = run_scaled(p, "dense", None)
    assert int(p.d_flags) == dk.FLAG_BLOCK_RANGE and bool(torch.isfinite(out.float()).all())
    p.d_flags.zero_()
    p.d_ctx[1] = 1000
    run_scaled(p, "dense", None)
    assert int(p.d_flags) == dk.FLAG_LENGTH


def test_scaled_attention_on_another_stream_and_in_a_graph(kernel):
    p = ScaledProblem(9, (500, 40), (9, 20), 16, 2, 128, 16).cuda()
    want = run_scaled(p, "causal", None)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    out, lse = run_scaled(p, "causal", None, stream=stream)
    stream.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = run_scaled(p, "causal", None)
    for k in range(2):
        p.d_scales[:, :, 1] += 1
        graph.replay()
        torch.cuda.synchronize()
        want = run_scaled(p, "causal", None)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_scaled_attention_expired_waits_report_a_timeout(monkeypatch):
    """The producers copy nothing: every wait runs out, and the next call is right again."""
    monkeypatch.setenv("DSPARK_TREE_ATTN_KERNEL", "tc")
    p = ScaledProblem(10, (500, 40), (9, 20), 16, 2, 128, 16).cuda()
    monkeypatch.setenv("DSPARK_TEST_HOLD_NS", "2000000")
    run_scaled(p, "dense", None)
    torch.cuda.synchronize()
    assert int(p.d_flags) == dk.FLAG_TIMEOUT
    monkeypatch.delenv("DSPARK_TEST_HOLD_NS")
    p.d_flags.zero_()
    out, lse = run_scaled(p, "dense", None)
    want, z, to, tl = attention(p, "dense", None)
    close(out, want, to)
    assert int(p.d_flags) == 0


def test_scaled_attention_tail_behind_a_heavy_token(kernel):
    """20,000 tokens with 0.1% of the weight between them, behind one that has the rest: their share is not lost."""
    D, n = 128, 20001
    p = ScaledProblem(11, (n,), (1,), 4, 1, D, 16, k_exp=(0, 1), v_exp=(0, 1))
    j = torch.arange(n + 1)
    page, off = p.table[0].long()[j // 16], j % 16
    rows = torch.zeros((n + 1, 2 * D))
    rows[0, 0] = 16.0           # the heavy token's key
    rows[1:, D:] = 1.0          # the others' values; the heavy one's are 0
    p.cache[page, 0, off] = rows.to(torch.float8_e4m3fn).view(torch.uint8)
    p.qkv[:] = 0
    p.qkv[:, :, 0] = (math.log(n) + math.log(1000.0)) / 16.0 * D ** 0.5
    check_scaled(p, "dense", None)


def test_scaled_attention_nan_codes(kernel):
    """NaN codes of drafted tokens reach only the rows that see them."""
    p = ScaledProblem(7, (100,), (6,), 8, 2, 128, 16)
    for j in (102, 104):
        p.cache[int(p.table[0, j // 16]), :, j % 16, 128 + j % 7::9] = 0x7f if j == 102 else 0xff
    check_scaled(p, "causal", None)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,nq", [(1, 17), (4, 8), (3, 11), (4, 16), (5, 13)])
def test_scaled_attention_row_groups(D, G, nq, kernel):
    """17 to 65 rows a KV head: contexts of no token, of one tile, over several CTAs; requests of fewer rows."""
    ctx, tokens = (0, 64, 1, 2500, 130), (nq, nq, nq, nq, nq)
    p = ScaledProblem(G + nq, ctx, tokens, 2 * G, 2, D, 16, packed=True)
    check_scaled(p, "tree", tree_mask(tokens, 1, D, empty=(0, nq)))
    tokens = (2 * nq - 1, 0, 1, nq, nq)
    p = ScaledProblem(G + nq + 1, ctx, tokens, 2 * G, 2, D, 24)
    check_scaled(p, "causal", None)


@pytest.mark.parametrize("D,G,nq", [(256, 2, 3), (128, 8, 4), (64, 6, 9), (128, 4, 16), (256, 8, 7)])
def test_scaled_attention_row_groups_with_empty_rows_bad_pages_and_rows_behind(D, G, nq, kernel):
    """A row that sees nothing, rows behind the last sequence, then a page out of range: as if its tokens were not there."""
    tokens = (nq, nq - 1)
    p = ScaledProblem(D + nq, (0, 150), tokens, 2 * G, 2, D, 16, pad_rows=3).cuda()
    mask, n = tree_mask(tokens, 1, D, empty=(0, nq)), sum(tokens)
    mask = torch.cat([mask, torch.full((3, 1), -1, dtype=torch.int64)])
    out = torch.full((n + 3, 2 * G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 3, 2 * G), 7.0, device="cuda")
    run_scaled(p, "tree", mask, out=out, lse=lse)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all()) and bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())
    want, z, to, tl = attention(p, "tree", mask)
    close(out[:n], want, to)
    assert int(p.d_flags) == 0
    # the third page of the second request: its 16 tokens are left out
    p.d_table[1, 2] = -1
    got = run_scaled(p, "tree", mask)
    assert int(p.d_flags) == dk.FLAG_BLOCK_RANGE
    p.d_flags.zero_()
    fresh = p.d_cache.clone()
    page = int(p.table[1, 2])
    p.d_table[1, 2] = page
    p.d_cache[page] = 0        # V of 0, and scores of 0: they count for the sum only
    zeros = run_scaled(p, "tree", mask)
    p.d_cache.copy_(fresh)
    # e^lse of both, 16 tokens of e^0 apart (lse below 2^4, off by some 2^-20 of it; out twice rounded to bf16, 2^-8 each)
    a, b = got[1][nq:n].double().exp(), zeros[1][nq:n].double().exp()
    assert ((b - a - 16).abs() <= 2.0 ** -12 * b).all()
    assert ((got[0][nq:n].double() * (a / b)[..., None] - zeros[0][nq:n].double()).abs() <= 2.0 ** -6 * got[0][nq:n].double().abs().max()).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq", [5, 12])
def test_scaled_attention_rising_scores(D, nq, kernel):
    """A maximum that grows by less and by more than an octave a tile, down to the last token; and one that falls."""
    n = 1500
    for k, last in enumerate((1.0, 30.0, -60.0)):
        p = ScaledProblem(12 + k, (n,), (nq,), 4, 1, D, 16, k_exp=(-4, -3), v_exp=(-2, 3))
        j = torch.arange(n + nq)
        page, off = p.table[0].long()[j // 16], j % 16
        p.cache[page, 0, off, :16] = (j / (n + nq) * 256)[:, None].expand(-1, 16).to(torch.float8_e4m3fn).view(torch.uint8)
        p.qkv[:, :, :16] = last * D ** 0.5 / 256
        check_scaled(p, "causal", None)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq", [1, 5, 12, 20])
def test_scaled_attention_of_huge_scores_stays_finite(D, nq, kernel):
    """Scores (base 2) around 2^20 to 2^26 that grow by 4 to 24 a tile: weights stay in fp16's range, equal values come out."""
    n, c = 900, D ** -0.5 / math.log(2.0)  # what a product of q and k counts in octaves
    for size in (2.0 ** 20, 1.3 * 2.0 ** 25, -1.1 * 2.0 ** 26):
        for step in (4, 12, 16, 24):
            p = ScaledProblem(13, (n,), (nq,), 4, 1, D, 16, k_exp=(0, 1), v_exp=(0, 1))
            j = torch.arange(n + nq)
            page, off = p.table[0].long()[j // 16], j % 16
            rows = torch.zeros((n + nq, 2 * D))
            rows[:, 0], rows[:, 1], rows[:, D:] = 256.0, (j // 64).float(), 1.0
            p.cache[page, 0, off] = rows.to(torch.float8_e4m3fn).view(torch.uint8)
            p.qkv[:] = 0
            p.qkv[:, :, 0], p.qkv[:, :, 1] = size / 256 / c, step / c
            p.cuda()
            out, lse = run_scaled(p, "dense", None)
            # weights rounded to fp16 (2^-11 each, one way at most) against their own sum, then out to bf16
            assert bool(torch.isfinite(lse).all()) and bool(((out.float() - 1).abs() <= 2.0 ** -8 + 2.0 ** -10).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq", [5, 12])
def test_scaled_attention_nan_codes_and_a_tail_of_more_rows(D, nq, kernel):
    """As above for 20 and 48 rows: NaN codes of drafted tokens, and a thin tail behind a heavy token."""
    p = ScaledProblem(7, (100, 3000), (nq, nq), 8, 2, D, 16)
    for b, c in enumerate((100, 3000)):
        for j in (c + 2, c + 4):
            p.cache[int(p.table[b, j // 16]), :, j % 16, D + j % 7::9] = 0x7f if j % 4 else 0xff
    check_scaled(p, "causal", None)
    n = 6001
    p = ScaledProblem(11, (n,), (nq,), 4, 1, D, 16, k_exp=(0, 1), v_exp=(0, 1))
    j = torch.arange(n + nq)
    page, off = p.table[0].long()[j // 16], j % 16
    rows = torch.zeros((n + nq, 2 * D))
    rows[0, 0] = 16.0
    rows[1:, D:] = 1.0
    p.cache[page, 0, off] = rows.to(torch.float8_e4m3fn).view(torch.uint8)
    p.qkv[:] = 0
    p.qkv[:, :, 0] = (math.log(n) + math.log(1000.0)) / 16.0 * D ** 0.5
    check_scaled(p, "dense", None)


# ------------------------------------------------------------------ one step after another


def test_a_loop_of_steps():
    """Insert, attention, verification, compaction and pages, three steps of a batch: what each place of the
    cache holds is the token that was accepted there, encoded; lengths and pages follow."""
    g = gen(12)
    B, H, D, bs, V, n, cols, pool = 4, 2, 64, 8, 200, 6, 16, 70
    live = Pool(B, cols, pool, bs)
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    pages, refs = ints([0] * B), ints([0] * pool)
    cache, scales = torch.full((pool, H, bs, 2 * D), 0x7f, dtype=torch.uint8, device="cuda"), torch.zeros((pool, H, 2), dtype=torch.int8, device="cuda")
    lens = ints([0, 3, 8, 21])
    f = flag()
    held = [torch.randn((x, H, 2 * D), generator=g).bfloat16() for x in lens.tolist()]  # what the cache should hold
    dk.resize_kv(table, pages, lens, refs, bs, error_flags=f)
    live.resize(lens.tolist())
    ctx_kv = torch.cat(held).cuda()
    start = [0, 0, 3, 11, 32]
    dk.insert_kv_scaled(ctx_kv[..., :D], ctx_kv[..., D:], cache, scales, table, ints(start), ints([0] * B), error_flags=f)
    rows_of = n + 1
    start = torch.arange(0, B * rows_of + 1, rows_of, dtype=torch.int32)
    up = torch.tensor([0, 0, 0, 1, 1, 2, 3] * B, dtype=torch.int32)
    for step in range(3):
        dk.resize_kv(table, pages, lens + rows_of, refs, bs, error_flags=f)
        live.resize((lens + rows_of).tolist())
        assert table.tolist() == live.table and refs.tolist() == live.refs
        kv = (torch.randn((B * rows_of, H, 2 * D), generator=g) * (1 + 40 * (step == 1))).bfloat16()
        d = kv.cuda()
        dk.insert_kv_scaled(d[..., :D], d[..., D:], cache, scales, table, start.cuda(), lens, error_flags=f)
        q = torch.randn((B * rows_of, 4, D), generator=g).bfloat16().cuda()
        out, _ = dk.tree_attention(q, cache, table, start.cuda(), lens, causal=True, block_scales=scales, error_flags=f)
        assert bool(torch.isfinite(out.float()).all())
        t, dr = probabilities(B * rows_of, V, g), probabilities(B * rows_of, V, g)
        t = (t + dr) / 2
        tok, u = torch.multinomial(dr[(torch.arange(B * rows_of) // rows_of) * rows_of + up], 1, generator=g)[:, 0], torch.rand(B * rows_of, generator=g)
        tokens, rows, counts = dk.verify_drafts(t.cuda(), tok.cuda(), start.cuda(), u.cuda(), 3, dr.cuda(), up.cuda(), error_flags=f)
        want = verify(t, dr, tok, start, up, u, 3, True)
        assert torch.equal(tokens.cpu(), want[0]) and torch.equal(rows.cpu(), want[1])
        old = lens.tolist()
        lens = dk.compact_kv(cache, table, lens, rows, counts, block_scales=scales, error_flags=f)
        for b in range(B):
            path = [0] + [int(x) for x in rows[b] if x >= 0]
            held[b] = torch.cat([held[b], kv[b * rows_of:(b + 1) * rows_of][path]])
            assert lens.tolist()[b] == old[b] + len(path) == held[b].shape[0]
        dk.resize_kv(table, pages, lens, refs, bs, error_flags=f)
        live.resize(lens.tolist())
        assert table.tolist() == live.table and refs.tolist() == live.refs and pages.tolist() == live.pages
        for b in range(B):
            j = torch.arange(held[b].shape[0])
            page = table.cpu()[b].long()[j // bs]
            got = value(cache.cpu()[page, :, j % bs], scales.cpu()[page])
            e = scales.cpu()[page].double().exp2().repeat_interleave(D, -1)
            # rounded once to a code and once more each time its page's scale grew or it moved: the largest scale
            # counts, half a step of 2^-3 relative or of the least code's 2^-9 each time
            assert ((got - held[b].double()).abs() <= 2.0 ** -4 * held[b].double().abs() * 1.07 + 4 * 2.0 ** -10 * e).all()
    assert int(f) == 0


def test_a_step_in_a_graph():
    """The whole step captured once and replayed: nothing of it asks for a length on the host."""
    g = gen(13)
    B, H, D, bs, V, n, cols, pool = 3, 2, 128, 16, 1000, 4, 8, 40
    kv, q = torch.randn((B * (n + 1), H, 2 * D), generator=g).bfloat16().cuda(), torch.randn((B * (n + 1), 4, D), generator=g).bfloat16().cuda()
    t, dr = probabilities(B * (n + 1), V, g).cuda(), probabilities(B * (n + 1), V, g).cuda()
    tok, u = torch.randint(0, V, (B * (n + 1),), generator=g).cuda(), torch.zeros(B * (n + 1), device="cuda")
    start = torch.arange(0, B * (n + 1) + 1, n + 1, dtype=torch.int32).cuda()

    def state():
        return dict(table=torch.full((B, cols), -1, dtype=torch.int32, device="cuda"), pages=ints([0] * B), refs=ints([0] * pool),
                    cache=torch.zeros((pool, H, bs, 2 * D), dtype=torch.uint8, device="cuda"),
                    scales=torch.zeros((pool, H, 2), dtype=torch.int8, device="cuda"), lens=ints([0] * B))

    def step(s):
        dk.resize_kv(s["table"], s["pages"], s["lens"] + n + 1, s["refs"], bs)
        dk.insert_kv_scaled(kv[..., :D], kv[..., D:], s["cache"], s["scales"], s["table"], start, s["lens"])
        out, _ = dk.tree_attention(q, s["cache"], s["table"], start, s["lens"], causal=True, block_scales=s["scales"])
        tokens, rows, counts = dk.verify_drafts(t, tok, start, u, n, dr)
        s["lens"].copy_(dk.compact_kv([s["cache"]], s["table"], s["lens"], rows, counts, block_scales=[s["scales"]]))
        dk.resize_kv(s["table"], s["pages"], s["lens"], s["refs"], bs)
        return out, tokens

    a, b = state(), state()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(state())
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step(b)
    torch.cuda.synchronize()
    for k in range(4):
        u.copy_(torch.rand(u.shape, generator=g))
        want = step(a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.equal(a[x], b[x]) for x in a)
    assert int(a["lens"].min()) >= 4


# ------------------------------------------------------------------ verification: residuals to the unit, long pieces, shares


def test_verify_residuals_to_the_unit():
    """After two rejections S = 1 + Z lies between two fp32 numbers, so S q has a rest of more than half a step of its
    fp32 part: what is left of an entry is the whole number of 2^-46 next to p - S q all the same, never below 0."""
    def one(p, q, u, want):
        P, Q = torch.zeros((3, 16)), torch.zeros((3, 16))
        for i, x in p.items():
            P[0, i] = float.fromhex(x)
        for i, x in q.items():
            Q[0, i] = float.fromhex(x)
        # token 9, which the target never has, is drafted twice and rejected twice
        got = check_verify(P, Q, torch.tensor([0, 9, 9]), torch.tensor([0, 3], dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                           torch.tensor([u, 0.5, 0.5]), 2)
        assert got[0].tolist() == [[want, -1, -1]]

    # entry 0 keeps 0.021 of 0.92, 5 and 13 the rest: the border between 0 and 5 lies just below these numbers
    p = {0: "0x1.d7e1cap-1", 5: "0x1.e6502ep-5", 13: "0x1.e2697p-11"}
    q = {0: "0x1.7f3488p-1", 5: "0x1.eb851ep-6", 9: "0x1.99999ap-3"}
    for u in ("0x1.dac448p-2", "0x1.dac44ap-2"):
        one(p, q, float.fromhex(u), 5)
    # entry 0 keeps less than half a unit: no number draws it
    p = {0: "0x1.f034b2p-24", 5: "0x1.6p-1", 13: "0x1.000928p-12"}
    q = {0: "0x1.8ce31ap-24", 5: "0x1.cp-2", 9: "0x1p-1"}
    for u in (0.125, 0.5, 0.875):
        one(p, q, u, 5)
    one(p, q, 1 - 2.0 ** -12, 13)


def test_verify_outputs_between_rows_and_over_inputs():
    """Outputs may lie in the gaps between rows of probabilities; over an input they are refused."""
    g = gen(21)
    t, d, tok, start, _, u = draws(100, [3, 2], g)
    wide = torch.full((t.shape[0], 120), float("nan"), device="cuda")
    wide[:, :100] = t.cuda()
    flat, base = wide.view(torch.int32).flatten(), (wide[:, :100], tok.cuda(), start.cuda(), u.cuda(), 3, d.cuda())
    counts, rows = flat[2 * 120 + 100:2 * 120 + 102], flat[3 * 120 + 114:4 * 120].view(2, 3)
    got = dk.verify_drafts(*base, counts=counts, rows=rows)
    assert all(torch.equal(x.cpu(), y) for x, y in zip(got, verify(t, d, tok, start, None, u, 3, True))) and got[2] is counts
    for over in (dict(counts=flat[2 * 120 + 99:2 * 120 + 101]), dict(rows=flat[3 * 120 + 115:4 * 120 + 1].view(2, 3)), dict(counts=base[2][1:]),
                 dict(counts=base[3].view(torch.int32)[:2]), dict(rows=rows, counts=rows[1, 1:])):
        with pytest.raises(dk.DSparkError, match="overlap"):
            dk.verify_drafts(*base, **over)


@pytest.mark.parametrize("replacement", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V,n", [(20, 131073, 5), (200, 9001, 5), (24, 70000, 7)])
def test_verify_trees_of_long_pieces(B, V, n, dtype, replacement):
    """More entries per warp than are kept in shared memory: every round reads its rows again."""
    g = gen(B + n)
    t, d, tok, start, up, u = draws(V, [n] * B, g, arity=4, distinct=not replacement, target_dtype=dtype, draft_dtype=dtype)
    u = 1 - (1 - u) * 0.4  # more rejections
    u[start[:-1].long()] = torch.rand(B, generator=g)
    got = check_verify(t, d, tok, start, up, u, 3, replacement)
    # requests whose last row has rejected two children and more: S is neither 0 nor 1 there
    lost = 0
    for b in range(B):
        k = int(got[2][b])
        at = int(got[1][b, k - 1]) if k else 0
        lost += k < 3 and int((up[start[b] + 1:start[b + 1]] == at).sum()) >= 2
    assert lost >= B // 4


SHARES = [  # p, q, their denominator, the fewest equal steps of u_0, u_1 and u_2 with all borders of tests and draws on a step
    ("replacement", (5, 2, 4, 5), (4, 8, 1, 3), 16, (4, 4, 3)), ("replacement", (3, 10, 1, 2), (2, 1, 12, 1), 16, (138, 12, 11)),
    ("distinct", (3, 2, 4, 3), (2, 8, 1, 1), 12, (4, 4, 3)), ("distinct", (10, 3, 1, 2), (2, 11, 2, 1), 16, (99, 22, 9)),
    ("taken", (3, 3, 3, 1), None, 10, (84, 10, 21)), ("taken", (1, 1, 1, 1), None, 4, (6, 4, 3))]


@pytest.mark.parametrize("kind,p,q,n,steps", SHARES)
def test_verify_shares_are_the_target_s(kind, p, q, n, steps):
    """Two children of one row: over the middles of all steps the first token comes exactly as often as the target has it, summed
    over the drafts by how often these are drawn; for drafts taken without drawing, whatever they are."""
    V = len(p)
    u = torch.cartesian_prod(*[(torch.arange(k) + 0.5) / k for k in steps])
    B, total = u.shape[0], torch.zeros(V, dtype=torch.float64)
    P = (torch.tensor(p) / n).expand(3 * B, V).contiguous().cuda()
    Q = None if q is None else (torch.tensor(q) / n).expand(3 * B, V).contiguous().cuda()
    up, start = torch.zeros(3 * B, dtype=torch.int32, device="cuda"), torch.arange(0, 3 * B + 1, 3, dtype=torch.int32, device="cuda")
    for x in range(V):
        for y in range(V):
            if kind == "distinct" and x == y:
                continue
            tok = torch.tensor([0, x, y]).repeat(B).cuda()
            tokens, _, _ = dk.verify_drafts(P, tok, start, u.flatten().cuda(), 1, Q, up, replacement=kind != "distinct")
            share = torch.bincount(tokens[:, 0].cpu(), minlength=V).double() / B
            if kind == "taken":
                assert (share - torch.tensor(p).double() / n).abs().max() < 1e-12, (x, y, share)
            else:
                total += share * q[x] / n * (q[y] / n if kind == "replacement" else q[y] / (n - q[x]))
    assert kind == "taken" or (total - torch.tensor(p).double() / n).abs().max() < 1e-12, total


# ------------------------------------------------------------------ compaction and the pool at more than one turn of the threads


@pytest.mark.parametrize("bs,D,H", [(16, 256, 9), (3, 128, 33), (16, 64, 40)])
def test_compact_scaled_columns_in_turns(bs, D, H):
    """More 16-byte columns than a CTA has threads, of page-scaled caches: each turn has exponents of its own."""
    assert H * D // 8 > 256
    check_compact("scaled", [0, 5, 9, 14, 15, 16, 200], PATHS, H, D, bs)


def test_compact_scaled_columns_in_turns_of_a_long_path():
    """The same with more moves into one page than are looked up at once."""
    check_compact("scaled", [3, 70], [list(range(2, 1202, 2)), list(range(300, 900))], 17, 128, 400, layers=1)


@pytest.mark.parametrize("pages,n,free", [(8193, 1025, 8193), (70001, 4096, 70001), (8193, 4096, 2000), (70001, 4096, 1200), (5000, 1500, 800)])
def test_pool_fork_over_several_ctas(pages, n, free):
    """Pools of one, two and eight CTAs, more pairs than a CTA has threads, some of them in need of a page; pages that run
    out behind pair 1,024."""
    src = 5
    live = Live(n + src, 40, pages, 2, layers=1, H=1)
    lens = [79, 1, 16, 33, 0]
    live.resize([2 * 40, 2, 16, 40, 3] + [0] * n)
    live.check()
    if free < pages:  # the others are held by somebody else
        r = random.Random(n)
        left = [p for p, x in enumerate(live.ref.refs) if x == 0]
        for p in r.sample(left, len(left) - free):
            live.ref.refs[p] = 1
        live.refs.copy_(ints(live.ref.refs))
    live.set_lens(lens + [0] * n)
    order = list(range(src, n + src))
    random.Random(pages).shuffle(order)
    live.fork([((i * 7 + i // 5) % src, d) for i, d in enumerate(order)])
    need = sum(lens[(i * 7 + i // 5) % src] % 2 for i in range(n))
    assert need > 512 and (free >= need or free > 1024 * need // n)
    live.check(0 if free >= need else dk.FLAG_PAGES)
    assert sum(live.ref.pages[d] > 0 for d in order) > 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq", [1, 5, 12, 20])
def test_scaled_attention_of_the_lowest_scores(D, nq, kernel):
    """Every score (base 2) within a few percent of fp32's lowest number, all alike: the mean of the values comes out."""
    n, c = 200, D ** -0.5 / math.log(2.0)  # what a product of q and k counts in octaves
    p = ScaledProblem(14, (n,), (nq,), 4, 1, D, 16, k_exp=(0, 1), v_exp=(0, 1))
    j = torch.arange(n + nq)
    page, off = p.table[0].long()[j // 16], j % 16
    rows = torch.zeros((n + nq, 2 * D))
    rows[:, 0] = 256.0
    rows[:, D:] = (j % 8)[:, None].float()
    p.cache[page, 0, off] = rows.to(torch.float8_e4m3fn).view(torch.uint8)
    p.qkv[:] = 0
    p.qkv[:, :, 0] = -3.2e38 / 256 / c
    assert 3.1e38 < abs(float(p.qkv[0, 0, 0])) * 256 * c < 3.3e38
    p.cuda()
    out, lse = run_scaled(p, "dense", None)
    # weights are alike (1 each) and the values whole: their sums are exact, the quotient rounded in fp32 and to bf16
    mean = float((j % 8).double().mean())
    assert bool(((out.double() - mean).abs() <= (2.0 ** -8 + 2.0 ** -21) * mean).all())
    assert bool(((lse / (float(p.qkv[0, 0, 0]) * 256 * D ** -0.5) - 1).abs() <= 2.0 ** -20).all())


# ------------------------------------------------------------------ far offsets, calls side by side


def test_scaled_cache_beyond_32_bits(kernel):
    """Insert, attention, compaction and fork in pages beyond 2^32 bytes of a cache do what they do in a small one."""
    g = gen(31)
    D, bs, H, nq = 128, 16, 8, 20
    small = ScaledProblem(15, (100, 30, 45), (nq, 3, 0), 2 * H, H, D, bs).cuda()
    pages = (1 << 32) // (H * bs * 2 * D) * 9 // 8
    shift = pages - small.blocks
    big, scales = torch.empty((pages, H, bs, 2 * D), dtype=torch.uint8, device="cuda"), torch.zeros((pages, H, 2), dtype=torch.int8, device="cuda")
    big[shift:], scales[shift:] = small.d_cache, small.d_scales
    near, far = (small.d_cache, small.d_scales, small.d_table), (big, scales, torch.where(small.d_table >= 0, small.d_table + shift, -1).to(torch.int32))
    assert int(far[2][0].max()) * H * bs * 2 * D > 1 << 32
    kv, f = torch.randn((nq + 3, 2, H, D), generator=g).bfloat16().cuda(), flag()
    rows, counts = ints([[2, 5, 9, 17], [2, -1, -1, -1], [-1] * 4]), ints([4, 1, 0])
    got = []
    for cache, sc, table in (near, far):
        dk.insert_kv_scaled(kv[:, 0], kv[:, 1], cache, sc, table, small.d_start, small.d_ctx, error_flags=f)
        out = dk.tree_attention(small.d_q, cache, table, small.d_start, small.d_ctx, causal=True, block_scales=sc, error_flags=f)
        lens = dk.compact_kv(cache, table, small.d_ctx, rows, counts, block_scales=sc, error_flags=f)
        got.append((*out, lens, cache[-small.blocks:], sc[-small.blocks:]))
    assert int(f) == 0 and all(torch.equal(a, b) for a, b in zip(*got))
    # request 0 continued as a fourth: the one free page, beyond 2^32 bytes, takes its last tokens
    free = max(set(range(shift, pages)) - set(far[2].flatten().tolist()))
    assert free * H * bs * 2 * D > 1 << 32
    table, refs = torch.full((4, far[2].shape[1]), -1, dtype=torch.int32, device="cuda"), torch.ones(pages, dtype=torch.int32, device="cuda")
    table[:3], refs[free] = far[2], 0
    lens = torch.cat([lens, ints([0])])
    full, tail = divmod(int(lens[0]), bs)
    old = int(table[0, full])
    dk.fork_kv(big, table, -(-lens // bs), lens, ints([0]), ints([3]), refs, block_scales=scales, error_flags=f)
    assert tail and int(table[3, full]) == free and int(refs[free]) == 1 and int(lens[3]) == int(lens[0]) and int(f) == 0
    assert torch.equal(big[free, :, :tail], big[old, :, :tail]) and torch.equal(scales[free], scales[old])


def test_verify_rows_beyond_32_bits():
    """Requests whose rows of probabilities lie beyond 2^32 bytes."""
    g = gen(32)
    t, d, tok, start, up, u = draws(131072, [3, 4, 2], g, arity=2)
    T, far = t.shape[0], 9000
    wide = [torch.empty((far + T, 131072), device="cuda") for _ in range(2)]
    tokens, parents, numbers = torch.zeros(far + T, dtype=torch.int64), torch.zeros(far + T, dtype=torch.int32), torch.zeros(far + T)
    for x, y in zip((*wide, tokens, parents, numbers), (t, d, tok, up, u)):
        x[far:] = y
    assert far * 131072 * 4 > 1 << 32
    got = dk.verify_drafts(wide[0], tokens.cuda(), (start + far).cuda(), numbers.cuda(), 4, wide[1], parents.cuda())
    assert all(torch.equal(x.cpu(), y) for x, y in zip(got, verify(t, d, tok, start, up, u, 4, True)))


def test_calls_side_by_side_on_two_streams():
    """Each operator in two graphs replayed at once on different streams, between calls on a third: no call shares anything with another."""
    g = gen(33)
    p = ScaledProblem(16, (900, 33, 400), (7, 20, 3), 16, 2, 128, 16).cuda()
    t, d, tok, start, up, u = [x.cuda() for x in draws(5000, [9, 20, 5], g, arity=3)]
    kv = torch.randn((30, 2, 2, 128), generator=g).bfloat16().cuda()

    def state():
        return dict(cache=p.d_cache.clone(), scales=p.d_scales.clone(), table=torch.full((6, 70), -1, dtype=torch.int32, device="cuda"),
                    pages=ints([0] * 6), refs=ints([0] * p.blocks), lens=ints([40, 7, 0, 0, 0, 0]))

    def work(s):
        a = dk.tree_attention(p.d_q, s["cache"], p.d_table, p.d_start, p.d_ctx, causal=True, block_scales=s["scales"])
        b = dk.verify_drafts(t, tok, start, u, 8, d, up)
        dk.resize_kv(s["table"], s["pages"], s["lens"], s["refs"], 16)
        dk.fork_kv([s["cache"]], s["table"], s["pages"], s["lens"], ints_src, ints_dst, s["refs"], block_scales=[s["scales"]])
        dk.insert_kv_scaled(kv[:, 0], kv[:, 1], s["cache"], s["scales"], p.d_table, p.d_start, p.d_ctx)
        return *a, *b

    ints_src, ints_dst = ints([0, 1, 0, 1]), ints([2, 3, 4, 5])
    first = state()
    want = work(first)
    torch.cuda.synchronize()
    streams, states, graphs, outs = [torch.cuda.Stream() for _ in range(3)], [state() for _ in range(2)], [], []
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(work(s))
        graphs.append(graph)
    for turn in range(3):
        fresh = state()
        for s in states:
            for k, x in state().items():
                s[k].copy_(x)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            third = work(fresh)
        torch.cuda.synchronize()
        for out, s in zip((*outs, third), (*states, fresh)):
            assert all(torch.equal(a, b) for a, b in zip(out, want)) and all(torch.equal(s[k], first[k]) for k in first)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 1.5])
def test_scaled_attention_takes_any_scale(D, scale, kernel):
    """Scales of none, of either sign, so small that products underflow, and large, over exponents far apart and near."""
    for nq, k_exp in ((3, (-6, -3)), (20, (-32, 3))):
        p = ScaledProblem(17 + nq, (150, 0, 70), (nq, 2, nq), 8, 2, D, 16, k_exp=k_exp)
        p.cuda()
        out, lse = run_scaled(p, "causal", None, scale=scale)
        want, z, to, tl = attention(p, "causal", None, scale=scale)
        close(lse, z, tl)
        close(out, want, to)
        assert int(p.d_flags) == 0


@pytest.mark.parametrize("D,nq", [(64, 1), (64, 4), (128, 1)])
def test_scaled_attention_calls_behind_one_another_lose_nothing(D, nq, monkeypatch):
    """Grids that fill the GPU, one call behind another: as fast, to a fifth, as launched without any overlap (a tenth of the CTAs that
    had to wait for a slot would cost a half), and the same bits."""
    g = torch.Generator(device="cuda").manual_seed(D)
    B, H, bs = 64, 8, 16
    ctx = [1024 + 7168 * i // (B - 1) for i in range(B)]
    need = [-(-(c + nq) // bs) for c in ctx]
    table, order, at = torch.zeros((B, max(need)), dtype=torch.int32, device="cuda"), torch.randperm(sum(need), generator=g, device="cuda").int(), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = torch.randint(0, 0x70, (at, H, bs, 2 * D), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(-9, -6, (at, H, 2), generator=g, device="cuda").to(torch.int8)
    q = torch.randn((B * nq, 8 * H, D), generator=g, device="cuda").bfloat16()
    start, lens = torch.arange(0, B * nq + 1, nq, dtype=torch.int32, device="cuda"), ints(ctx)
    graphs, outs = [], []
    for early in ("1", "0"):
        monkeypatch.setenv("DSPARK_PDL", early)
        dk.tree_attention(q, cache, table, start, lens, causal=True, block_scales=scales)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(8):
                out = dk.tree_attention(q, cache, table, start, lens, causal=True, block_scales=scales)
        graphs.append(graph)
        outs.append(out)
    times = [[], []]
    for _ in range(12):
        for graph, t in zip(graphs, times):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            t.append(a.elapsed_time(b))
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    assert min(times[0]) < 1.2 * min(times[1]), (min(times[0]), min(times[1]))
