"""Plain 64-bit forms of the draft-attention operators and their input
recipes, for the tests (no arithmetic is shared with the library)."""

import math
import random

import torch

SEED = 20460


def gen(seed):
    g = torch.Generator()
    g.manual_seed(SEED + seed)
    return g


class Problem:
    """A paged cache with the requests' tokens in shuffled blocks; every other
    byte of it is 0xFF (NaN in bf16 and in e4m3)."""

    def __init__(self, seed, ctx, nq, Hq, Hkv, D, bs, fp8, extra_blocks=3, pad_rows=0, packed=False, table_cols=None,
                 q_std=2.0, device="cuda"):
        g = gen(seed)
        self.ctx, self.nq, self.Hq, self.Hkv, self.D, self.bs, self.fp8 = list(ctx), list(nq), Hq, Hkv, D, bs, fp8
        B = len(ctx)
        need = [-(-(c + n) // bs) for c, n in zip(ctx, nq)]
        self.blocks = sum(need) + extra_blocks
        order = torch.randperm(self.blocks, generator=g)
        cols = table_cols or max(1, max(need))
        self.table = torch.full((B, cols), -7, dtype=torch.int32)  # entries past a length are not read
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.cache = torch.full((self.blocks, Hkv, bs, 2 * D * (1 if fp8 else 2)), 0xFF, dtype=torch.uint8)
        self.cache = self.cache if fp8 else self.cache.view(torch.bfloat16)
        self.k_scale, self.v_scale = torch.tensor([0.037]), torch.tensor([0.021])
        T = sum(nq)
        x = torch.randn((T + pad_rows, Hq + (2 * Hkv if packed else 0), D), generator=g) * q_std
        self.qkv = x.to(torch.bfloat16)
        self.start = torch.tensor([sum(nq[:b]) for b in range(B + 1)], dtype=torch.int32)
        self.T = T
        for b in range(B):
            n = ctx[b] + nq[b]
            k, v = torch.randn((n, Hkv, D), generator=g), torch.randn((n, Hkv, D), generator=g)
            self.write(b, torch.arange(n), k, v)
        self.device = device

    def write(self, b, j, k, v):
        blk, off = self.table[b].long()[j // self.bs], j % self.bs
        if self.fp8:
            row = torch.cat([(k / self.k_scale).clamp(-448, 448), (v / self.v_scale).clamp(-448, 448)], -1)
            self.cache[blk, :, off] = row.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            self.cache[blk, :, off] = torch.cat([k, v], -1).to(torch.bfloat16)

    def rows(self, b, n=None):
        """(K, V) [n, Hkv, D] of request b in 64 bits."""
        j = torch.arange(self.ctx[b] + self.nq[b] if n is None else n)
        r = self.cache[self.table[b].long()[j // self.bs], :, j % self.bs]
        if self.fp8:
            r = r.view(torch.float8_e4m3fn).double()
            return r[..., :self.D] * self.k_scale.double(), r[..., self.D:] * self.v_scale.double()
        return r[..., :self.D].double(), r[..., self.D:].double()

    def cuda(self):
        """The call's tensors on the device."""
        d = self.device
        self.d_cache, self.d_table, self.d_start = self.cache.to(d), self.table.to(d), self.start.to(d)
        self.d_ctx = torch.tensor(self.ctx, dtype=torch.int32, device=d)
        self.d_q = self.qkv.to(d)[:, :self.Hq]
        self.d_ks, self.d_vs = (self.k_scale.to(d), self.v_scale.to(d)) if self.fp8 else (None, None)
        self.d_flags = torch.zeros(1, dtype=torch.int32, device=d)
        return self

    def scale_kw(self):
        return dict(k_scale=self.d_ks, v_scale=self.d_vs)


def tree_mask(nq, words, seed, empty=()):
    """Random trees: a node sees itself and its ancestors; rows in `empty` see nothing."""
    r = random.Random(SEED + seed)
    rows = []
    for n in nq:
        seen = []
        for i in range(n):
            up = r.randrange(-1, i) if i else -1
            seen.append((seen[up] if up >= 0 else 0) | (1 << i))
        rows += seen
    for t in empty:
        rows[t] = 0
    out = torch.zeros((len(rows), words), dtype=torch.int64)
    for t, m in enumerate(rows):
        for w in range(words):
            x = (m >> (64 * w)) & ((1 << 64) - 1)
            out[t, w] = x - (1 << 64) if x >= 1 << 63 else x
    return out


def seen_of(p, b, kind, mask):
    """[nq, ctx + nq] truth values."""
    n, Q = p.ctx[b], p.nq[b]
    tail = torch.ones((Q, Q), dtype=torch.bool)
    if kind == "causal":
        tail = tail.tril()
    elif kind == "tree":
        lo = int(p.start[b])
        for i in range(Q):
            for j in range(Q):
                tail[i, j] = bool((int(mask[lo + i, j // 64]) >> (j % 64)) & 1)
    return torch.cat([torch.ones((Q, n), dtype=torch.bool), tail], 1)


def attention(p, kind, mask, scale=None):
    """(out, lse, tol_out, tol_lse): the definition in 64 bits, and how far 32-bit
    sums of rounded weights may be from it.

    With u = 2^-8 half a bf16 step and w = u (2^-11 with fp8: fp16 weights): the
    weights are rounded once, sum |v| of them with relative error w each; the
    result is rounded once (u).  Scores are sums of D exact products in 32 bits
    (tensor cores may truncate: 2^-22 an addition), so a score is off by d =
    scale (D + 8) 2^-22 sum |q k|, fp16 queries by 2^-24 of the row's largest
    per element more; a weight by e^2d - 1.  Statistics and sums of n tiles cost
    n 2^-22, exponential and division 2^-21 each.
    """
    u, w = 2.0 ** -8, 2.0 ** -11 if p.fp8 else 2.0 ** -8
    scale = p.D ** -0.5 if scale is None else scale
    G = p.Hq // p.Hkv
    out = torch.zeros((p.T, p.Hq, p.D), dtype=torch.float64)
    lse = torch.full((p.T, p.Hq), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(p.ctx)):
        lo, hi = int(p.start[b]), int(p.start[b + 1])
        if hi == lo:
            continue
        k, v = p.rows(b)
        seen = seen_of(p, b, kind, mask)
        q = p.qkv[lo:hi, :p.Hq].double()
        for h in range(p.Hq):
            kh, vh = k[:, h // G], v[:, h // G]
            x = torch.where(seen, (q[:, h] @ torch.nan_to_num(kh, nan=0.0, posinf=0.0, neginf=0.0).T) * scale, -math.inf)
            bad = ~torch.isfinite(kh).all(1)
            if (seen & bad).any():
                full = (q[:, h, None, :] * kh[None]).sum(-1) * scale
                x = torch.where(seen & bad, full, x)
            z = torch.logsumexp(x, 1)
            wt = torch.where(seen, (x - z[:, None]).exp(), 0.0)
            wt = torch.where((z == -math.inf)[:, None], torch.zeros_like(wt), wt)
            # only what is seen is summed
            o = torch.stack([(wt[i, seen[i]][:, None] * vh[seen[i]]).sum(0) for i in range(hi - lo)])
            fine = torch.nan_to_num(kh.abs(), nan=0.0, posinf=0.0)
            d = abs(scale) * 2.0 ** -22 * ((p.D + 8) * (q[:, h].abs() @ fine.T).amax(1, keepdim=True)
                                      + (2.0 ** -2 * q[:, h].abs().amax(1, keepdim=True) * fine.sum(1).amax() if p.fp8 else 0.0))
            A = wt @ torch.nan_to_num(vh.abs(), nan=0.0, posinf=0.0, neginf=0.0)
            steps = (kh.shape[0] // 64 + 80) * 2.0 ** -22
            out[lo:hi, h], lse[lo:hi, h] = o, z
            to[lo:hi, h] = u * o.abs() * (1 + u) + (w + 2.1 * d + steps) * A * (1 + u) + 1e-30
            tl[lo:hi, h] = (d[:, 0] + steps + z.abs() * 2.0 ** -22).nan_to_num(nan=math.inf, posinf=math.inf)
    return out, lse, to, tl


def close(got, want, tol):
    """Everything within tol; infinities and NaN where they belong."""
    got, want = got.double().cpu(), want.cpu()
    same = (got == want) | (got.isnan() & want.isnan())
    off = (got - want).abs()
    ok = same | (off <= tol)
    assert ok.all(), f"{(~ok).sum()} of {ok.numel()} off, worst {float((off / tol)[~ok].max())} times the tolerance, " \
                     f"first at {torch.nonzero(~ok)[0].tolist()}: {got[~ok][0]} for {want[~ok][0]}"


def weight(p, lse, weights, decay, scale=None):
    """(weights, tolerance) after one accumulation with this (32-bit) lse."""
    scale = p.D ** -0.5 if scale is None else scale
    G = p.Hq // p.Hkv
    out, tol = weights.double().clone(), torch.zeros(weights.shape, dtype=torch.float64)
    for b, n in enumerate(p.ctx):
        lo, hi = int(p.start[b]), int(p.start[b + 1])
        k, _ = p.rows(b, n)
        add, t = torch.zeros((p.Hkv, n), dtype=torch.float64), torch.zeros((p.Hkv, n), dtype=torch.float64)
        for h in range(p.Hq):
            q = p.qkv[lo:hi, h].double()
            kh = k[:, h // G]
            x = (q @ kh.T) * scale
            z = lse[lo:hi, h].double().cpu()[:, None]
            pw = torch.where(z == -math.inf, torch.zeros_like(x), (x - z).exp())
            d = abs(scale) * 2.0 ** -22 * ((p.D + 8) * (q.abs() @ kh.abs().T)
                                      + (0.25 * q.abs().amax(1, keepdim=True) * kh.abs().sum(1) if p.fp8 else 0.0))
            add[h // G] += pw.sum(0)
            t[h // G] += (pw * (1.1 * d + (x.abs() + z.abs().nan_to_num(posinf=0.0) + 8) * 2.0 ** -22)).sum(0)
        rows = (hi - lo) * G
        out[b, :, :n] = decay * out[b, :, :n] + add
        tol[b, :, :n] = t + (rows + 4) * 2.0 ** -23 * out[b, :, :n].abs() + 1e-30
    return out, tol


def evict(p_cache, table, bs, ctx, weights, pos, seen, budget, sinks, recent):
    """(cache, weights, positions, lens) after the eviction, by sorting."""
    cache, w, po = p_cache.clone(), weights.clone(), pos.clone()
    lens = []
    for b, n in enumerate(ctx):
        lens.append(min(n, budget))
        if n <= budget:
            continue
        for h in range(weights.shape[1]):
            def rank(j):
                x, at = float(weights[b, h, j]), int(pos[b, h, j])
                kept = at < sinks or at >= seen[b] - recent
                return (0 if kept else 1, 0.0 if kept else (math.inf if x != x else -x), 1 if (x != x and not kept) else 0, j)
            order = sorted(range(n), key=rank)
            keep = set(order[:budget])
            holes = [j for j in range(budget) if j not in keep]
            movers = [j for j in range(budget, n) if j in keep]
            w[b, h, budget:n], po[b, h, budget:n] = 0.0, -1
            for d, s in zip(holes, movers):
                w[b, h, d], po[b, h, d] = weights[b, h, s], pos[b, h, s]
                cache[int(table[b, d // bs]), h, d % bs] = p_cache[int(table[b, s // bs]), h, s % bs]
    return cache, w, po, lens
