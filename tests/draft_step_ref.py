"""Plain 64-bit forms of the draft-step operators, for the tests (no arithmetic
is shared with the library)."""

import math

import numpy as np
import torch

from draft_attn_ref import Problem, gen

EXP_MIN, EXP_MAX = -32, 31


# ------------------------------------------------------------------ verification


def clean(x):
    x = x.double().numpy().copy()
    x[np.isnan(x)] = 0.0
    return np.clip(x, 0.0, 1.0)


def verify(target, draft, tokens, start, parents, u, max_accepted, replacement):
    """(tokens, rows, counts) by the walk as it is defined, each rejection on the whole distribution."""
    B, V = start.numel() - 1, target.shape[1]
    ot = torch.full((B, max_accepted + 1), -1, dtype=torch.int64)
    orow = torch.full((B, max_accepted), -1, dtype=torch.int32)
    oc = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        lo, n = int(start[b]), int(start[b + 1] - start[b])
        if n == 0:
            continue
        uu = [min(max(0.0, float(x)) if x == x else 0.0, 1.0) for x in u[lo:lo + n]]
        at, steps = 0, []
        while True:
            p = clean(target[lo + at])
            R, Z, taken = p.copy(), 1.0, None
            q = None if draft is None else clean(draft[lo + at])
            lost = []
            kids = [i for i in range(1, n) if (i - 1 if parents is None else int(parents[lo + i])) == at] if len(steps) < max_accepted else []
            for i in kids:
                x = int(tokens[lo + i])
                known = 0 <= x < V
                if q is None:
                    if not Z > 0:
                        break
                    r = R[x] if known else 0.0
                    if uu[i] * Z < r:
                        taken = i
                        break
                    Z -= r
                    if known:
                        R[x] = 0.0
                    continue
                left = 1.0 if replacement else 1.0 - sum(q[y] for y in lost)
                if not left > 2.0 ** -24 or not Z > 0:
                    break
                if known and uu[i] * (q[x] / left) * Z < R[x]:
                    taken = i
                    break
                now = q.copy()
                if not replacement:
                    now[lost] = 0.0
                R = np.maximum(R - Z * (now / left), 0.0)
                if known:
                    lost.append(x)
                    if not replacement:
                        R[lost] = 0.0
                Z = R.sum()
            if taken is None:
                break
            steps.append(taken)
            at = taken
        if not R.sum() > 0:
            R = p
        oc[b] = len(steps)
        for j, i in enumerate(steps):
            ot[b, j], orow[b, j] = tokens[lo + i], i
        if R.sum() > 0:
            cum = np.cumsum(R)
            ot[b, len(steps)] = min(int(np.searchsorted(cum, uu[0] * cum[-1], side="right")), int(np.flatnonzero(R)[-1]))
    return ot, orow, oc


# ------------------------------------------------------------------ page-scaled caches


def value(codes, e):
    """Codes [..., 2 D] with exponents [..., 2], in 64 bits."""
    D = codes.shape[-1] // 2
    return codes.view(torch.float8_e4m3fn).double() * torch.ldexp(torch.ones(e.shape).double(), e.int()).repeat_interleave(D, -1)


def encode(x, e):
    """x [..., 2 D] over 2^e as codes (saturating)."""
    D = x.shape[-1] // 2
    y = x * torch.ldexp(torch.ones(e.shape).double(), -e.int()).repeat_interleave(D, -1)
    return y.clamp(-448, 448).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)


def grow(codes, was, e):
    """A page's codes [H, n, 2 D] from exponents `was` [H, 2] to `e`."""
    D = codes.shape[-1] // 2
    keep = (was == e).repeat_interleave(D, -1)[:, None]
    return torch.where(keep, codes, encode(value(codes, was[:, None]), e[:, None]))


def exponent(x):
    """The least e with |x| <= 448 2^e for the finite x of a [H, n, D], in [-32, 31]: [H]."""
    out = []
    for h in range(x.shape[0]):
        top = x[h][torch.isfinite(x[h])].abs().max().item() if torch.isfinite(x[h]).any() else 0.0
        e = EXP_MIN
        while e < EXP_MAX and math.ldexp(448.0, e) < top:
            e += 1
        out.append(e)
    return torch.tensor(out, dtype=torch.int8)


def insert_scaled(k, v, cache, scales, table, start, ctx, bs):
    """(cache, scales) after the insert; requests and pages out of range are left out."""
    cache, scales = cache.clone(), scales.clone()
    for b in range(len(ctx)):
        lo, n = int(start[b]), int(start[b + 1] - start[b])
        j = 0
        while j < n:
            blk, off = divmod(ctx[b] + j, bs)
            m, page = min(bs - off, n - j), int(table[b, blk])
            if 0 <= page < cache.shape[0]:
                kk, vv = (t[lo + j:lo + j + m].double().transpose(0, 1) for t in (k, v))
                e = torch.stack([exponent(kk), exponent(vv)], 1)
                if off:
                    e = torch.maximum(e, scales[page])
                    cache[page, :, :off] = grow(cache[page, :, :off], scales[page], e)
                x = torch.cat([kk, vv], -1)
                cache[page, :, off:off + m] = encode(x, e[:, None])
                scales[page] = e
            j += m
    return cache, scales


def compact(caches, scales, table, ctx, rows, counts, first, bs):
    """(caches, scales, lens) after the accepted rows have moved."""
    caches, blocks = [c.clone() for c in caches], caches[0].shape[0]
    scales = None if scales is None else [s.clone() for s in scales]
    lens = []
    for b in range(len(ctx)):
        k = int(counts[b])
        path = [int(x) for x in rows[b, :max(0, k)]]
        room = table.shape[1] * bs
        if (ctx[b] < 0 or k < 0 or k > rows.shape[1] or ctx[b] + first + k > room or any(r < first + j for j, r in enumerate(path))
                or any(a >= z for a, z in zip(path, path[1:])) or any(ctx[b] + r >= room for r in path)):
            lens.append(ctx[b])
            continue
        lens.append(ctx[b] + first + k)
        moves = [(ctx[b] + r, ctx[b] + first + j) for j, r in enumerate(path) if r != first + j]
        moves = [m for m in moves if all(0 <= int(table[b, x // bs]) < blocks for x in m)]
        for layer, cache in enumerate(caches):
            before = cache.clone()
            if scales is None:
                for s, d in moves:
                    cache[int(table[b, d // bs]), :, d % bs] = before[int(table[b, s // bs]), :, s % bs]
                continue
            was = scales[layer].clone()
            for blk in sorted({d // bs for _, d in moves}):
                page, into = int(table[b, blk]), [m for m in moves if m[1] // bs == blk]
                e = torch.stack([was[page]] + [was[int(table[b, s // bs])] for s, _ in into]).amax(0)
                cache[page] = grow(before[page], was[page], e)
                for s, d in into:
                    p = int(table[b, s // bs])
                    cache[page, :, d % bs] = grow(before[p, :, s % bs][:, None], was[p], e)[:, 0]
                scales[layer][page] = e
    return caches, scales, lens


class ScaledProblem(Problem):
    """A page-scaled cache in the place of a per-tensor one: the same codes with random exponents."""

    def __init__(self, seed, ctx, nq, Hq, Hkv, D, bs, k_exp=(-6, -3), v_exp=(-8, 8), **kw):
        super().__init__(seed, ctx, nq, Hq, Hkv, D, bs, True, **kw)
        g = gen(seed + 77)
        self.scales = torch.stack([torch.randint(lo, hi, (self.blocks, Hkv), generator=g) for lo, hi in (k_exp, v_exp)], -1).to(torch.int8)

    def rows(self, b, n=None):
        j = torch.arange(self.ctx[b] + self.nq[b] if n is None else n)
        page = self.table[b].long()[j // self.bs]
        x = value(self.cache[page, :, j % self.bs], self.scales[page])
        return x[..., :self.D], x[..., self.D:]

    def cuda(self):
        super().cuda()
        self.d_scales = self.scales.to(self.device)
        return self


# ------------------------------------------------------------------ the pool


class Pool:
    """Block table rows, reference counts and lengths, by one page at a time."""

    def __init__(self, rows, width, pages, bs):
        self.table = [[-1] * width for _ in range(rows)]
        self.pages, self.lens, self.refs, self.bs, self.width = [0] * rows, [0] * rows, [0] * pages, bs, width
        self.copies = []

    def take(self):
        for p, n in enumerate(self.refs):
            if n == 0:
                self.refs[p] = 1
                return p
        return None

    def fork(self, pairs):
        """The sound pairs, in order; the copies (old page, new page, tokens) they make."""
        R, done = len(self.table), []
        held = list(self.pages)
        for i, (s, d) in enumerate(pairs):
            if not (0 <= s < R and 0 <= d < R) or held[d] != 0 or any(x == d for x, _ in pairs) or any(y == d for _, y in pairs[:i]):
                continue
            full, tail = divmod(self.lens[s], self.bs)
            if self.lens[s] < 0 or held[s] > self.width or self.lens[s] > held[s] * self.bs:
                continue
            if tail and not 0 <= self.table[s][full] < len(self.refs):
                continue
            done.append((s, d, full, tail))
        fresh = []
        free = [p for p, n in enumerate(self.refs) if n == 0]
        for s, d, full, tail in done:
            if tail and not free:
                continue
            fresh.append((s, d, full, tail, free.pop(0) if tail else None))
        for s, d, full, tail, page in fresh:
            for k in range(full):
                self.table[d][k] = self.table[s][k]
                if 0 <= self.table[s][k] < len(self.refs):
                    self.refs[self.table[s][k]] += 1
            if tail:
                self.table[d][full] = page
                self.refs[page] = 1
                self.copies.append((self.table[s][full], page, tail))
            self.pages[d], self.lens[d] = full + (tail > 0), self.lens[s]

    def resize(self, tokens):
        want = [-(-t // self.bs) for t in tokens]
        ok = [0 <= self.pages[r] <= self.width and tokens[r] >= 0 and want[r] <= self.width for r in range(len(want))]
        for r in range(len(want)):
            while ok[r] and self.pages[r] > want[r]:
                self.pages[r] -= 1
                p = self.table[r][self.pages[r]]
                self.table[r][self.pages[r]] = -1
                if 0 <= p < len(self.refs) and self.refs[p] > 0:
                    self.refs[p] -= 1
        free, asked = self.refs.count(0), 0
        for r in range(len(want)):
            need = max(0, want[r] - self.pages[r]) if ok[r] else 0
            asked += need
            if need and asked <= free:
                for _ in range(need):
                    self.table[r][self.pages[r]] = None  # taken below, lowest first
                    self.pages[r] += 1
        for row in self.table:
            for k, p in enumerate(row):
                if p is None:
                    row[k] = self.take()
