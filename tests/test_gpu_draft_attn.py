"""The draft-attention operators on the GPU against their definitions in 64
bits: the cos|sin table, rotary positions with the K/V insert, the drafted
tokens' attention, the accumulated attention weight, the eviction, and a run
of them together.  Tolerances: draft_attn_ref.py and beside each test."""

import decimal
import math

import pytest
import torch

import speculative_decoding_draft_ctx_gb300 as dk
from draft_attn_ref import Problem, attention, close, evict, gen, tree_mask, weight

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the table

PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")


def cos_sin(pos, f):
    """cos and sin of pos * f with f the double, the turns taken off exactly."""
    with decimal.localcontext() as c:
        c.prec = 70
        turns = decimal.Decimal(pos) * decimal.Decimal(f) / (2 * PI)
        a = float((turns - turns.to_integral_value()) * 2 * PI)
    return math.cos(a), math.sin(a)


TABLES = [(16, 1e4, None, 0, 5), (64, 1e6, None, 131000, 7), (2, 1e4, None, (1 << 31) - 3, 3), (6, 5e5, dict(kind="linear", factor=8), 1 << 20, 4),
          (128, 1e4, dict(kind="by_parts", factor=4, original_positions=4096), 65535, 3),
          (64, 5e5, dict(kind="bands", factor=8, original_positions=8192), 1 << 24, 3), (256, 1e4, None, 1, 1), (512, 1e4, None, 7, 2)]


@pytest.mark.parametrize("r,theta,scaling,first,count", TABLES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_table(r, theta, scaling, first, count, dtype):
    got = dk.rope_table(count, r, theta=theta, scaling=scaling, first_position=first, dtype=dtype).double().cpu()
    f, amp = dk.rope_frequencies(r, theta, scaling)
    for p in range(count):
        for i in range(r // 2):
            want = cos_sin(first + p, f[i])
            # the fixed-point frequency: 3 roundings of 2^-53 of it and 2^-64 of a turn, p times; the reduced angle
            # and its cosine 2^-23 each, the product 2^-24; then one rounding to bf16
            tol = amp * ((first + p) * (f[i] * 2.0 ** -51 + 2.0 ** -61) + 2.0 ** -22)
            for x, y in zip(want, (got[p, i], got[p, r // 2 + i])):
                assert abs(float(y) - amp * x) <= tol + (2.0 ** -8 * (abs(amp * x) + tol) if dtype is torch.bfloat16 else 0.0)


def test_table_into_out_and_what_the_write_reads():
    out = torch.full((9, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    assert dk.rope_table(9, 32, theta=1e6, out=out) is out
    assert (out[0, :16] == 1).all() and (out[0, 16:] == 0).all()
    assert dk.rope_table(0, 32, out=out[:0]).shape == (0, 32)
    import workloads as wk

    wl = wk.WORKLOADS[1]
    recipe = wk.generate(wl.with_(num_ctx=8, pad_count=0)).cos_sin
    mine = dk.rope_table(recipe.shape[0], wl.rotary_dim, theta=wl.rope_theta).cpu()
    # both within half a bf16 step of the cosine: at most one step apart
    steps = (mine.view(torch.int16).int() - torch.as_tensor(recipe).view(torch.bfloat16).view(torch.int16).int()).abs()
    near_zero = (mine.float().abs() < 2.0 ** -12)
    assert (steps[~near_zero] <= 1).all()


# ------------------------------------------------------------------ the rotation


def rope_reference(x, table, pos, r, layout, inverse):
    """(the rotation in 64 bits, its tolerance): a bf16 rounding (2^-8) of fp32 sums of products."""
    x = x.double()
    row = table.double()[pos.clamp(0, table.shape[0] - 1)][:, None]
    c, s = row[..., :r // 2], row[..., r // 2:] * (-1 if inverse else 1)
    a = torch.arange(r // 2) * (2 if layout == "interleaved" else 1)
    b = a + (1 if layout == "interleaved" else r // 2)
    y, mag = x.clone(), x.abs()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
    mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    out_of = (pos < 0) | (pos >= table.shape[0])
    y[out_of], mag[out_of] = x[out_of], 0.0
    return y, 2.0 ** -8 * y.abs() + 2.0 ** -22 * mag


ROPES = [  # T, Hq, Hkv, D, r, layout, bs, fp8, inverse, fp32 table, odd strides
    (1, 1, 1, 64, 2, "half", 1, False, False, False, False),
    (7, 64, 8, 128, 64, "half", 16, False, False, False, False),
    (7, 5, 5, 128, 64, "interleaved", 16, True, True, True, False),
    (33, 6, 3, 128, 18, "half", 7, True, False, False, False),
    (33, 6, 3, 128, 18, "interleaved", 7, False, False, True, False),
    (5, 3, 1, 256, 256, "half", 32, True, False, True, False),
    (5, 3, 1, 256, 50, "interleaved", 5, False, True, False, True),
    (19, 8, 2, 64, 64, "half", 48, True, False, False, True),
    (600, 12, 4, 64, 16, "half", 16, False, False, False, False),
    (1300, 2, 1, 128, 32, "interleaved", 64, True, False, False, False),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,r,layout,bs,fp8,inverse,fp32,odd", ROPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_kv_insert(T, Hq, Hkv, D, r, layout, bs, fp8, inverse, fp32, odd, in_place):
    g = gen(T + D + r)
    W = (Hq + 2 * Hkv) * D + (3 if odd else 0)  # 3 more: rows no longer 16-byte aligned
    qkv = (torch.randn((T, W), generator=g) * 2).to(torch.bfloat16)
    pos = torch.randint(0, 97, (T,), generator=g)
    slots = torch.randperm(T * 2 + bs, generator=g)[:T]
    if T > 4:
        slots[2], pos[1], pos[3], slots[4] = -1, 97, -1, (T * 2 // bs + 2) * bs  # padding; outside the table; outside the cache
    table = dk.rope_table(97, r, dtype=torch.float32 if fp32 else torch.bfloat16).cpu()
    blocks = T * 2 // bs + 2
    cache = torch.full((blocks, Hkv, bs, 2 * D * (1 if fp8 else 2)), 0xFF, dtype=torch.uint8)
    cache = cache if fp8 else cache.view(torch.bfloat16)
    ks, vs = torch.tensor([0.11]), torch.tensor([0.07])
    d = qkv.cuda()
    first = 1 if odd else 0
    q, k, v = (d[:, a:a + n * D].unflatten(1, (n, D)) for a, n in ((first, Hq), (first + Hq * D, Hkv), (first + (Hq + Hkv) * D, Hkv)))
    ref = [x.cpu().clone() for x in (q, k, v)]
    dcache, flags = cache.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = dk.rope_kv_insert(q, k, table.cuda(), pos.cuda(), r, v=v, layout=layout, inverse=inverse, slot_mapping=slots.cuda(), kv_cache=dcache,
                               k_scale=ks.cuda(), v_scale=vs.cuda(), error_flags=flags, **(dict(q_out=q, k_out=k) if in_place else {}))
    assert not in_place or (qo is q and ko is k)
    for got, x in ((qo, ref[0]), (ko, ref[1])):
        close(got, *rope_reference(x, table, pos, r, layout, inverse))
    assert torch.equal(v.cpu(), ref[2])
    if in_place and odd:
        assert torch.equal(d[:, 0].cpu(), qkv[:, 0]) and torch.equal(d[:, -2:].cpu(), qkv[:, -2:])
    # the cache: exactly the rounded K' and V of the tokens with a slot, every other byte untouched
    kp = ko.cpu()
    live = (slots >= 0) & (slots < blocks * bs) & (pos >= 0) & (pos < 97)
    if fp8:
        enc = lambda x, s: (x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        row = torch.cat([enc(kp, ks), enc(ref[2], vs)], -1)
    else:
        row = torch.cat([kp, ref[2]], -1)
    at = slots[live]
    cache[at // bs, :, at % bs] = row[live]
    assert torch.equal(dcache.cpu().view(torch.uint8), cache.view(torch.uint8))
    assert int(flags) == (dk.FLAG_POS_RANGE | dk.FLAG_SLOT_RANGE if T > 4 else 0)


def test_rope_without_insert_and_empty():
    x = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
    table = dk.rope_table(8, 64)
    pos = torch.tensor([0, 5, 7], device="cuda")
    q, k = dk.rope_kv_insert(x, x[:, :1], table, pos, 64)
    close(q, *rope_reference(x.cpu(), table.cpu(), pos.cpu(), 64, "half", False))
    assert torch.equal(k, q[:, :1])
    assert torch.equal(q[0], x[0])  # position 0
    q, k = dk.rope_kv_insert(x[:0], x[:0, :1], table, pos[:0], 64)
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient(layout):
    """The inverse rotation is the gradient: against the formula, and against differences of a 64-bit form."""
    g = gen(5)
    T, H, D, r = 4, 2, 64, 36
    x = torch.randn((T, H, D), generator=g).to(torch.bfloat16)
    up = torch.randn((T, H, D), generator=g).to(torch.bfloat16)
    table, pos = dk.rope_table(64, r, dtype=torch.float32), torch.tensor([0, 9, 33, 63])
    dx, _ = dk.rope_kv_insert(up.cuda(), up[:, :1].cuda(), table, pos.cuda(), r, layout=layout, inverse=True)
    want, tol = rope_reference(up, table.cpu(), pos, r, layout, True)
    close(dx, want, tol)
    loss = lambda z: float((rope_reference(z, table.cpu(), pos, r, layout, False)[0] * up.double()).sum())  # noqa: E731
    for t, h, i in ((1, 0, 0), (2, 1, r - 1), (3, 0, r // 2), (1, 1, r + 3)):
        e = torch.zeros((T, H, D), dtype=torch.float64)
        e[t, h, i] = 1.0
        # linear in x: the difference is exact up to 64-bit rounding
        slope = (loss(x.double() + e) - loss(x.double() - e)) / 2
        assert abs(float(dx[t, h, i]) - slope) <= float(tol[t, h, i]) + 1e-9


# ------------------------------------------------------------------ attention


@pytest.fixture(params=["rule", "mma", "tc"])
def kernel(request, monkeypatch):
    """Each test runs with the kernel the call's sizes choose and with each one pinned."""
    if request.param != "rule":
        monkeypatch.setenv("DSPARK_TREE_ATTN_KERNEL", request.param)
    return request.param


ATTN = [  # ctx, nq, Hq, Hkv, D, bs, fp8, mask
    ((1,), (1,), 1, 1, 64, 1, False, "dense"),
    ((0,), (1,), 8, 8, 128, 16, False, "causal"),
    ((0, 3, 64, 63, 65), (1, 7, 2, 1, 3), 8, 2, 128, 16, False, "causal"),
    ((5, 0, 127, 700), (7, 5, 0, 7), 24, 8, 128, 16, False, "dense"),
    ((5, 0, 127, 700), (7, 5, 0, 7), 24, 8, 128, 48, True, "tree"),
    ((1000, 17), (1, 1), 32, 2, 128, 64, True, "dense"),
    ((333, 2, 0), (13, 40, 64), 6, 3, 64, 3, False, "tree"),
    ((333, 2, 0), (13, 40, 64), 6, 3, 64, 100, True, "causal"),
    ((200, 130), (9, 70), 16, 1, 256, 32, False, "tree"),
    ((200, 130), (9, 70), 5, 5, 256, 7, True, "tree"),
    ((64, 1), (1, 2), 2, 1, 256, 16, False, "dense"),
    ((31, 500), (3, 1), 16, 1, 64, 16, True, "dense"),
    ((2000,), (130,), 4, 4, 128, 16, False, "tree"),
    ((0, 0), (0, 0), 4, 4, 128, 16, False, "dense"),
    ((4000, 300), (64, 33), 32, 4, 128, 16, False, "tree"),
    ((3000, 0, 700), (64, 5, 20), 40, 8, 128, 64, True, "tree"),
    ((2500, 129), (30, 70), 20, 4, 64, 100, False, "causal"),
    ((2500, 127), (17, 70), 40, 4, 64, 16, True, "tree"),
    (tuple(range(0, 300)), tuple(i % 3 for i in range(300)), 2, 2, 64, 16, False, "causal"),
]


def run_attention(p, kind, mask, **kw):
    return dk.tree_attention(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, tree_mask=mask.cuda() if kind == "tree" else None,
                             causal=kind == "causal", error_flags=p.d_flags, **p.scale_kw(), **kw)


@pytest.mark.parametrize("ctx,nq,Hq,Hkv,D,bs,fp8,kind", ATTN)
def test_attention(ctx, nq, Hq, Hkv, D, bs, fp8, kind, kernel):
    p = Problem(len(ctx) + D + bs, ctx, nq, Hq, Hkv, D, bs, fp8, packed=True).cuda()
    mask = tree_mask(nq, max(1, -(-max(nq) // 64)), D, empty=(0,) if sum(nq) else ())
    out, lse = run_attention(p, kind, mask)
    want, z, to, tl = attention(p, kind, mask)
    close(lse, z, tl)
    close(out, want, to)
    assert int(p.d_flags) == 0


@pytest.mark.parametrize("D,fp8", [(64, False), (128, False), (128, True), (64, True), (256, True)])
def test_attention_many_small_items(D, fp8, kernel):
    """More (request, KV head) pairs than CTAs, of one and of two row tiles in turn: a CTA's state from item to item."""
    g = gen(D + fp8)
    nq = tuple(int(x) for x in torch.tensor([3, 6, 27, 30, 1, 40, 25, 26])[torch.randint(0, 8, (48,), generator=g)])
    ctx = tuple(int(x) for x in torch.tensor([0, 3, 40, 100, 120, 167, 200, 300])[torch.randint(0, 8, (48,), generator=g)])
    p = Problem(D, ctx, nq, 40, 8, D, 16, fp8).cuda()
    mask = tree_mask(nq, 1, D)
    out, lse = run_attention(p, "tree", mask)
    want, z, to, tl = attention(p, "tree", mask)
    close(lse, z, tl)
    close(out, want, to)
    assert int(p.d_flags) == 0


def test_attention_and_weight_more_requests_than_threads(kernel):
    """The search for a CTA's first request takes them in chunks of a CTA's threads."""
    n = 1500
    ctx, nq = [0 if i % 97 else i // 97 for i in range(n)], [(i % 11 == 0) * (1 + i % 3) for i in range(n)]
    ctx[-1], nq[-1] = 700, 20
    p = Problem(11, ctx, nq, 4, 2, 64, 16, False).cuda()
    out, lse = run_attention(p, "dense", None)
    want, z, to, tl = attention(p, "dense", None)
    close(lse, z, tl)
    close(out, want, to)
    w = torch.rand((n, 2, 701), generator=gen(1))
    d = w.cuda()
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, d, decay=0.5, error_flags=p.d_flags)
    close(d, *weight(p, lse, w, 0.5))
    assert int(p.d_flags) == 0


def test_attention_rows_without_anything_and_rows_behind(kernel):
    """A row that sees nothing: zeros and -inf.  Rows of no request and outputs behind them stay."""
    p = Problem(3, (0, 4), (3, 2), 4, 2, 128, 16, False, pad_rows=3).cuda()
    mask = torch.tensor([[0], [2], [0], [0], [3], [-1], [-1], [-1]])
    out = torch.full((8, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, 4), 6.0, device="cuda")
    assert run_attention(p, "tree", mask, out=out, lse=lse)[0] is out
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all() and (out[2] == 0).all() and (lse[2] == -math.inf).all()
    assert (out[5:] == 5).all() and (lse[5:] == 6).all()
    want, z, to, tl = attention(p, "tree", mask)
    close(lse[:5], z, tl)
    close(out[:5], want, to)
    # rows before the first request's, and between two
    p.d_start = torch.tensor([2, 5, 5], dtype=torch.int32, device="cuda")
    p.d_ctx = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    out.fill_(5.0)
    run_attention(p, "dense", mask, out=out, lse=lse)
    assert (out[:2] == 5).all() and (out[5:] == 5).all() and (out[2:5] != 5).any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctx", [3, 700])
def test_attention_keeps_what_is_masked_out(fp8, D, ctx, kernel):
    """NaN and infinities in drafted tokens reach the rows that see them and no others."""
    nq = (6, 40)
    p = Problem(D + ctx, (ctx, 70), nq, 4, 2, D, 16, fp8)
    mask = torch.zeros((46, 1), dtype=torch.int64)
    mask[:6, 0] = torch.tensor([1, 2, 4, 8, 17, 32])
    mask[6:, 0] = torch.tensor([1 << i for i in range(40)])
    for b, j, dim, x in ((0, 0, 5, math.nan), (0, 1, 7, math.inf), (0, 2, 9, -math.inf), (1, 39, 0, math.nan)):
        blk, off = int(p.table[b, (p.ctx[b] + j) // 16]), (p.ctx[b] + j) % 16
        if fp8:
            p.cache[blk, 1, off, D + dim] = 0x7F if b == 0 else 0xFF
        else:
            p.cache[blk, 1, off, D + dim] = x
    blk, off = int(p.table[0, (ctx + 3) // 16]), (ctx + 3) % 16
    p.cache[blk, 0, off, :D] = 0xFF if fp8 else math.nan  # K of token 3, KV head 0: its own row alone is NaN
    p.cuda()
    out, lse = run_attention(p, "tree", mask)
    want, z, to, tl = attention(p, "tree", mask)
    close(lse, z, tl)
    close(out, want, to)
    assert out.isnan().any() and out[4].isnan().any() and not out[5].isnan().any()
    assert torch.isfinite(out[6:45]).all()


def test_attention_infinite_context_value_and_large_scores(kernel):
    p = Problem(8, (90,), (2,), 2, 1, 128, 16, False, q_std=300.0)
    p.cache[int(p.table[0, 1]), 0, 3, 130] = math.inf
    p.cuda()
    mask = torch.tensor([[3], [3]])
    out, lse = run_attention(p, "tree", mask)
    want, z, to, tl = attention(p, "tree", mask)
    close(lse, z, tl)
    keep = [i for i in range(128) if i != 2]
    close(out[..., keep], want[..., keep], to[..., keep])
    assert not torch.isfinite(out[..., 2]).any()


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7])
def test_attention_any_scale(scale, kernel):
    p = Problem(4, (70, 5), (3, 9), 8, 2, 64, 16, True).cuda()
    out, lse = run_attention(p, "causal", None, scale=scale)
    want, z, to, tl = attention(p, "causal", None, scale=scale)
    close(lse, z, tl)
    close(out, want, to)


def test_attention_queries_of_any_magnitude_over_fp8(kernel):
    """Rows far above and below fp16's range: each row is scaled on its own."""
    p = Problem(6, (50,), (4,), 2, 1, 128, 16, True)
    p.qkv = (p.qkv.float() * torch.tensor([2.0 ** -130, 1e-12, 1.0, 1e30]).view(4, 1, 1)).to(torch.bfloat16)
    p.cuda()
    out, lse = run_attention(p, "dense", None)
    want, z, to, tl = attention(p, "dense", None)
    close(lse[:3], z[:3], tl[:3])
    close(out[:3], want[:3], to[:3])
    best = (p.qkv[3].double() @ p.rows(0)[0][:, 0].T).argmax(-1)  # e^(1e30 ...): one token takes all
    v = p.rows(0)[1][best, 0]
    close(out[3], v, 1.01 * 2.0 ** -8 * v.abs())


def test_attention_out_of_range_lengths_and_blocks(kernel):
    """Bad lengths leave the request out, bad blocks their tokens; nothing else changes."""
    def problem():
        return Problem(7, (40, 33, 50, 21), (3, 2, 4, 2), 4, 2, 128, 16, False, table_cols=5)
    p = problem().cuda()
    good_out, good_lse = run_attention(p, "dense", None)
    assert int(p.d_flags) == 0
    for what in ("start", "ctx", "negative", "mask"):
        q = problem().cuda()
        out, lse = torch.full_like(good_out, 3.0), torch.full_like(good_lse, 4.0)
        kind, mask = "dense", None
        gone = [3, 4]
        if what == "start":
            q.d_start[4] = 99  # request 3 ends behind the rows
            gone = [9, 10]
        elif what == "ctx":
            q.d_ctx[1] = 79  # 81 tokens in 80 places
        elif what == "negative":
            q.d_ctx[1] = -1
        else:
            q.d_start = torch.tensor([0, 3, 3, 3, 11], dtype=torch.int32, device="cuda")
            q.d_table[3, :5] = q.d_table[0, :5]
            q.d_ctx[3] = 0
            kind, mask = "tree", torch.full((11, 1), -1)
            run_attention(q, kind, mask, out=out, lse=lse)
            assert int(q.d_flags) == 0  # eight drafted tokens fit a word
            q = Problem(7, (4,), (65,), 2, 2, 128, 16, False).cuda()
            o2 = torch.full((65, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
            run_attention(q, "tree", torch.full((65, 1), -1), out=o2)
            assert int(q.d_flags) == dk.FLAG_LENGTH and (o2 == 3).all()
            continue
        run_attention(q, kind, mask, out=out, lse=lse)
        assert int(q.d_flags) == dk.FLAG_LENGTH, what
        rest = [t for t in range(11) if t not in gone]
        assert (out[gone] == 3).all() and (lse[gone] == 4).all()
        assert torch.equal(out[rest], good_out[rest]) and torch.equal(lse[rest], good_lse[rest])
    for entry in (-1, 10 ** 6):
        q = problem().cuda()
        q.d_table[2, 1] = entry  # tokens 16..31 of request 2
        out, lse = run_attention(q, "dense", None)
        assert int(q.d_flags) == dk.FLAG_BLOCK_RANGE
        rest = [t for t in range(11) if t not in (5, 6, 7, 8)]
        assert torch.equal(out[rest], good_out[rest])
        # the same as attention over the other tokens
        k, v = p.rows(2)
        keep = [j for j in range(54) if not 16 <= j < 32]
        r = Problem(7, (34,), (4,), 4, 2, 128, 16, False)
        r.write(0, torch.arange(38), k[keep].float(), v[keep].float())
        r.qkv = p.qkv[5:9].clone()
        want, z, to, tl = attention(r, "dense", None)
        close(lse[5:9], z, tl)
        close(out[5:9], want, to)


def test_attention_far_offsets_in_a_large_cache(kernel):
    """Rows beyond 2^31 elements of the cache."""
    D, bs, H = 128, 16, 8
    blocks = (1 << 31) // (H * bs * 2 * D) * 5 // 4
    p = Problem(9, (100, 30), (5, 2), 16, H, D, bs, False)
    used = sorted(set(p.table[p.table >= 0].tolist()))
    big = torch.empty((blocks, H, bs, 2 * D), dtype=torch.bfloat16, device="cuda")
    shift = blocks - p.blocks
    big[shift:] = p.cache.cuda()
    p.cuda()
    d_table = torch.where(p.d_table >= 0, p.d_table + shift, p.d_table)
    out, lse = dk.tree_attention(p.d_q, big, d_table, p.d_start, p.d_ctx)
    want, z, to, tl = attention(p, "dense", None)
    close(out, want, to)
    close(lse, z, tl)
    assert used and max(used) + shift > (1 << 31) // (H * bs * 2 * D)
    w = torch.zeros((2, H, 100), device="cuda")
    dk.accumulate_attention_weight(p.d_q, big, d_table, p.d_start, p.d_ctx, lse, w)
    close(w, *weight(p, lse, torch.zeros((2, H, 100)), 1.0))


def test_attention_same_bits_again_and_on_another_stream_and_in_graphs(kernel):
    p = Problem(12, (900, 20, 3000), (7, 7, 7), 16, 2, 128, 16, False).cuda()
    a = run_attention(p, "dense", None)
    b = run_attention(p, "dense", None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = run_attention(p, "dense", None, stream=s)
    d = run_attention(p, "dense", None, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(a[0], c[0]) and torch.equal(a[0], d[0])
    # two graphs replayed side by side on different streams, and eager calls between
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run_attention(p, "dense", None))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        e = run_attention(p, "dense", None)
    torch.cuda.synchronize()
    for o, z in outs + [e]:
        assert torch.equal(o, a[0]) and torch.equal(z, a[1])


# ------------------------------------------------------------------ the accumulated weight

WEIGHTS = [  # ctx, nq, Hq, Hkv, D, bs, fp8, decay
    ((1,), (1,), 1, 1, 64, 1, False, 1.0),
    ((70, 0, 5, 130), (7, 3, 0, 1), 16, 2, 128, 16, False, 0.9),
    ((70, 0, 5, 130), (7, 3, 0, 1), 15, 5, 128, 7, True, 0.0),
    ((64, 500), (40, 9), 8, 1, 64, 48, True, 1.0),
    ((300, 65), (66, 2), 2, 2, 256, 100, False, 0.5),
    ((300, 65), (3, 64), 12, 4, 256, 16, True, 1.0),
    ((700, 300, 1), (40, 33, 34), 16, 2, 128, 16, False, 0.7),
    ((300, 1500), (64, 33), 20, 2, 64, 32, True, 0.7),
    (tuple(range(0, 300)), tuple(i % 3 for i in range(300)), 2, 2, 64, 16, False, 0.5),
]


@pytest.mark.parametrize("ctx,nq,Hq,Hkv,D,bs,fp8,decay", WEIGHTS)
def test_weight(ctx, nq, Hq, Hkv, D, bs, fp8, decay):
    p = Problem(sum(ctx) + D, ctx, nq, Hq, Hkv, D, bs, fp8, packed=True).cuda()
    mask = tree_mask(nq, -(-max(max(nq), 1) // 64), 3)
    _, lse = run_attention(p, "tree", mask)
    places = max(ctx) + 5
    w = torch.rand((len(ctx), Hkv, places), generator=gen(1))
    d = w.cuda()
    assert dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, d, decay=decay, k_scale=p.d_ks,
                                          error_flags=p.d_flags) is d
    close(d, *weight(p, lse, w, decay))
    assert int(p.d_flags) == 0
    e = w.cuda()
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, e, decay=decay, k_scale=p.d_ks)
    assert torch.equal(d, e)


@pytest.mark.parametrize("D,fp8", [(64, True), (128, False), (128, True), (256, False)])
def test_weight_many_small_items(D, fp8):
    """More (request, KV head) pairs than CTAs, of no, one and two row groups in turn."""
    g = gen(D + fp8)
    nq = tuple(int(x) for x in torch.tensor([3, 6, 27, 60, 0, 40, 1, 26])[torch.randint(0, 8, (48,), generator=g)])
    ctx = tuple(int(x) for x in torch.tensor([0, 3, 40, 100, 128, 167, 200, 300])[torch.randint(0, 8, (48,), generator=g)])
    p = Problem(D, ctx, nq, 40, 8, D, 16, fp8).cuda()
    _, lse = run_attention(p, "tree", tree_mask(nq, 1, 3))
    w = torch.rand((48, 8, 305), generator=gen(1))
    d = w.cuda()
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, d, decay=0.75, k_scale=p.d_ks, error_flags=p.d_flags)
    close(d, *weight(p, lse, w, 0.75))
    assert int(p.d_flags) == 0

@pytest.mark.parametrize("D", [64, 128])
def test_weight_ragged_rows_over_fp8(D):
    """Heads of no, few and more rows than a group, several tiles and pairs per CTA, the same bits again."""
    nq = tuple((3, 6, 27, 60, 0, 1, 2, 19)[i % 8] for i in range(40))
    ctx = tuple((700, 3, 40, 1000, 128, 0, 2000, 300)[i * 5 % 8] for i in range(40))
    p = Problem(D + 1, ctx, nq, 20, 4, D, 16, True).cuda()
    _, lse = run_attention(p, "tree", tree_mask(nq, 1, 3))
    w = torch.rand((40, 4, 2003), generator=gen(1))
    d = w.cuda()
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, d, decay=0.75, k_scale=p.d_ks, error_flags=p.d_flags)
    close(d, *weight(p, lse, w, 0.75))
    assert int(p.d_flags) == 0
    e = w.cuda()
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, e, decay=0.75, k_scale=p.d_ks)
    assert torch.equal(d, e)


def test_weight_sums_to_the_rows_and_rows_without_anything():
    """Without drafted tokens seen, a head's weights sum to its rows; a row of lse -inf adds nothing."""
    p = Problem(2, (200,), (4,), 8, 2, 128, 16, False).cuda()
    mask = torch.zeros((4, 1), dtype=torch.int64)
    _, lse = run_attention(p, "tree", mask)
    w = torch.zeros((1, 2, 200), device="cuda")
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, w)
    assert (w.sum(-1).cpu() - 16.0).abs().max() < 1e-3
    lse[1] = -math.inf
    w.zero_()
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, w)
    assert (w.sum(-1).cpu() - 12.0).abs().max() < 1e-3


def test_weight_out_of_range():
    p = Problem(5, (40, 60), (2, 2), 4, 2, 64, 16, False).cuda()
    _, lse = run_attention(p, "dense", None)
    w = torch.ones((2, 2, 50), device="cuda")  # request 1 has 60 context tokens
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, w, error_flags=p.d_flags)
    assert int(p.d_flags) == dk.FLAG_LENGTH
    assert (w[1] == 1).all() and (w[0, :, :40] > 1).all() and (w[0, :, 40:] == 1).all()
    p.d_flags.zero_()
    p.d_table[0, 1] = -3
    w.fill_(1.0)
    p.d_ctx[1] = 45
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, w, error_flags=p.d_flags)
    assert int(p.d_flags) == dk.FLAG_BLOCK_RANGE
    assert (w[0, :, 16:32] == 1).all() and (w[0, :, :16] > 1).all()


# ------------------------------------------------------------------ eviction

EVICTS = [  # ctx, Hkv, D, bs, fp8, budget, sinks, recent, values
    ((1,), 1, 64, 1, False, 1, 0, 0, "rand"),
    ((2,), 1, 64, 16, False, 1, 0, 1, "rand"),
    ((100, 0, 33, 64), 2, 128, 16, False, 32, 4, 8, "rand"),
    ((100, 99, 33, 64), 3, 64, 7, True, 31, 0, 31, "ties"),
    ((300, 1000), 1, 256, 48, False, 200, 2, 3, "special"),
    ((5000, 20, 4097), 2, 128, 16, True, 2500, 4, 64, "ties"),
    ((20000,), 1, 64, 16, True, 700, 1, 16, "rand"),
]


@pytest.mark.parametrize("ctx,Hkv,D,bs,fp8,budget,sinks,recent,values", EVICTS)
@pytest.mark.parametrize("in_place", [True, False])
def test_evict(ctx, Hkv, D, bs, fp8, budget, sinks, recent, values, in_place):
    p = Problem(sum(ctx) + D, ctx, (0,) * len(ctx), Hkv, Hkv, D, bs, fp8).cuda()
    g = gen(budget)
    B, S = len(ctx), max(ctx) + 3
    w = torch.rand((B, Hkv, S), generator=g)
    if values == "ties":
        w = (w * 4).floor()
    elif values == "special":
        w = (w - 0.5) * 1e3
        w[:, :, ::7], w[:, :, 3::11], w[:, :, 5::13], w[:, :, 1::9], w[:, :, 2::9] = math.nan, math.inf, -math.inf, -0.0, 0.0
    pos = torch.stack([torch.stack([torch.randperm(S, generator=g) for _ in range(Hkv)]) for _ in range(B)]).to(torch.int32)
    seen = [max(1, c) for c in ctx]
    want = evict(p.cache, p.table, bs, ctx, w, pos, seen, budget, sinks, recent)
    dw, dp = w.cuda(), pos.cuda()
    kw = {} if in_place else dict(weights_out=torch.full_like(dw, 9.0), positions_out=torch.full_like(dp, 9))
    lens = dk.evict_kv(p.d_cache, p.d_table, p.d_ctx, dw, dp, torch.tensor(seen, dtype=torch.int32, device="cuda"), budget, sinks, recent,
                       error_flags=p.d_flags, **kw)
    assert lens.tolist() == want[3] and int(p.d_flags) == 0
    ow, op = (dw, dp) if in_place else (kw["weights_out"], kw["positions_out"])
    assert torch.equal(ow.cpu().view(torch.int32), want[1].view(torch.int32))
    assert torch.equal(op.cpu(), want[2])
    assert torch.equal(p.d_cache.cpu().view(torch.uint8), want[0].view(torch.uint8))
    if not in_place:
        assert torch.equal(dw.cpu().view(torch.int32), w.view(torch.int32)) and torch.equal(dp.cpu(), pos)


@pytest.mark.parametrize("what", ["weights_out", "positions_out"])
def test_evict_one_of_two_in_place(what):
    p = Problem(9, (600, 40, 700), (0, 0, 0), 2, 2, 64, 16, False).cuda()
    w, pos = torch.rand((3, 2, 705), generator=gen(2)), torch.arange(705, dtype=torch.int32).repeat(3, 2, 1)
    want = evict(p.cache, p.table, 16, (600, 40, 700), w, pos, [600, 40, 700], 300, 4, 8)
    dw, dp = w.cuda(), pos.cuda()
    out = torch.full_like(dw if what == "weights_out" else dp, 9)
    lens = dk.evict_kv(p.d_cache, p.d_table, p.d_ctx, dw, dp, torch.tensor([600, 40, 700], dtype=torch.int32, device="cuda"), 300, 4, 8,
                       error_flags=p.d_flags, **{what: out})
    assert lens.tolist() == want[3] and int(p.d_flags) == 0
    ow, op = (out, dp) if what == "weights_out" else (dw, out)
    assert torch.equal(ow.cpu(), want[1]) and torch.equal(op.cpu(), want[2])
    assert torch.equal(p.d_cache.cpu().view(torch.uint8), want[0].view(torch.uint8))
    kept = dw.cpu() if what == "weights_out" else dp.cpu()
    assert torch.equal(kept, w if what == "weights_out" else pos)


def test_evict_many_places_and_a_long_slice():
    """More places than the keys a CTA holds: one pair per cluster and many pairs."""
    for B, H, n, budget in ((1, 1, 300001, 100000), (160, 2, 17000, 16999)):
        bs, D = 64, 64
        blocks = B * -(-n // bs)
        table = torch.arange(blocks, dtype=torch.int32, device="cuda").flip(0).view(B, -1).contiguous()
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        w = torch.rand((B, H, n), generator=g, device="cuda")
        # the row holds its own number: what moved is read from the cache
        cache = torch.zeros((blocks, H, bs, 2 * D), dtype=torch.uint8, device="cuda")
        number = torch.arange(n, dtype=torch.int32, device="cuda")
        j = torch.arange(n, device="cuda")
        for b in range(B):
            rows = cache[table[b].long()[j // bs], :, j % bs].contiguous()
            rows.view(torch.int32)[..., 0] = number[:, None]
            cache[table[b].long()[j // bs], :, j % bs] = rows
        pos = number.expand(B, H, n).contiguous()
        lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
        out = dk.evict_kv(cache, table, lens, w, pos, lens, budget, sinks=3, recent=5)
        assert (out == budget).all()
        kept = torch.sort(pos[:, :, :budget], -1)[0]
        assert (kept[..., 1:] > kept[..., :-1]).all() and (pos[:, :, budget:] == -1).all() and (w[:, :, budget:] == 0).all()
        g.manual_seed(1)
        first = torch.rand((B, H, n), generator=g, device="cuda")
        first[:, :, :3], first[:, :, n - 5:] = 2.0, 2.0
        want = torch.sort(torch.sort(first, dim=-1, descending=True, stable=True)[1][:, :, :budget], -1)[0]
        assert torch.equal(kept.long(), want)
        for b in (0, B - 1):
            rows = cache[table[b].long()[j // bs], :, j % bs].contiguous().view(torch.int32)[..., 0]
            assert torch.equal(rows[:budget].T, pos[b, :, :budget])
        stay = pos[:, :, :budget] < budget
        assert torch.equal(pos[:, :, :budget][stay], number[:budget].expand(B, H, budget)[stay])


def test_evict_out_of_range():
    p = Problem(4, (40, 50, 60), (0, 0, 0), 2, 2, 64, 16, False).cuda()
    w = torch.rand((3, 2, 60), device="cuda")
    pos = torch.arange(60, dtype=torch.int32, device="cuda").expand(3, 2, 60).contiguous()
    seen = p.d_ctx.clone()
    before = [x.clone() for x in (p.d_cache, w, pos)]
    p.d_ctx[0], p.d_ctx[1], p.d_ctx[2] = 61, -1, 9  # too long, negative, within the budget
    lens = dk.evict_kv(p.d_cache, p.d_table, p.d_ctx, w, pos, seen, 10, error_flags=p.d_flags)
    assert int(p.d_flags) == dk.FLAG_LENGTH and lens.tolist() == [61, -1, 9]
    assert torch.equal(p.d_cache.view(torch.uint8), before[0].view(torch.uint8)) and torch.equal(w, before[1]) and torch.equal(pos, before[2])
    p.d_flags.zero_()
    p.d_ctx.copy_(seen)
    p.d_table[2, 0] = 10 ** 6
    dk.evict_kv(p.d_cache, p.d_table, p.d_ctx, w, pos, seen, 10, error_flags=p.d_flags)
    assert int(p.d_flags) == dk.FLAG_BLOCK_RANGE


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("fp8", [False, True])
def test_draft_step_with_eviction(fp8):
    """Table, rotation with insert, attention, accumulated weight, eviction, attention over what is left -- as a
    draft step runs them, eagerly and from one captured graph, against the same chain in 64 bits."""
    Hq, Hkv, D, bs, r = 8, 2, 128, 16, 64
    ctx, nq, budget = (90, 37, 120), (4, 7, 5), 60
    p = Problem(21, ctx, nq, Hq, Hkv, D, bs, fp8, packed=True).cuda()
    T, B = sum(nq), len(ctx)
    table = dk.rope_table(512, r, theta=1e6, scaling=dict(kind="by_parts", factor=4, original_positions=128))
    pos = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, nq)])
    slots = torch.cat([p.table[b].long()[torch.arange(c, c + n) // bs] * bs + torch.arange(c, c + n) % bs
                       for b, (c, n) in enumerate(zip(ctx, nq))])
    mask = tree_mask(nq, 1, 7)
    qkv = p.qkv.cuda()
    S = max(ctx)
    cache0 = p.d_cache.clone()
    d_pos, d_slots, d_mask, seen = pos.cuda(), slots.cuda(), mask.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda")
    token_pos0 = torch.arange(S, dtype=torch.int32, device="cuda").expand(B, Hkv, S).contiguous()
    w, token_pos = torch.zeros((B, Hkv, S), device="cuda"), token_pos0.clone()

    def step():
        q, k, v = (qkv[:, a:a + n] for a, n in ((0, Hq), (Hq, Hkv), (Hq + Hkv, Hkv)))
        q, k = dk.rope_kv_insert(q, k, table, d_pos, r, v=v, slot_mapping=d_slots, kv_cache=p.d_cache, k_scale=p.d_ks, v_scale=p.d_vs,
                                 error_flags=p.d_flags)
        out, lse = dk.tree_attention(q, p.d_cache, p.d_table, p.d_start, p.d_ctx, tree_mask=d_mask, error_flags=p.d_flags, **p.scale_kw())
        dk.accumulate_attention_weight(q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, w, k_scale=p.d_ks, error_flags=p.d_flags)
        lens = dk.evict_kv(p.d_cache, p.d_table, p.d_ctx, w, token_pos, seen, budget, sinks=2, recent=8, error_flags=p.d_flags)
        # the next step's drafted tokens: here one row per request over the shorter context
        rows = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        out2, lse2 = dk.tree_attention(q[:B], p.d_cache, p.d_table, rows, lens - 1, error_flags=p.d_flags, **p.scale_kw())
        return q, k, out, lse, lens, out2, lse2

    got = step()
    q, k, out, lse, lens, out2, lse2 = got
    assert int(p.d_flags) == 0 and lens.tolist() == [min(c, budget) for c in ctx]
    # attention over the cache as the insert left it (the insert itself: test_rope_kv_insert)
    p.qkv = torch.cat([q.cpu(), p.qkv[:, Hq:]], 1)
    ref = cache0.cpu()
    if fp8:
        enc = lambda x, s: (x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        row = torch.cat([enc(k.cpu(), p.k_scale), enc(qkv[:, Hq + Hkv:].cpu(), p.v_scale)], -1)
    else:
        row = torch.cat([k.cpu(), qkv[:, Hq + Hkv:].cpu()], -1)
    ref[slots // bs, :, slots % bs] = row
    p.cache = ref
    want, z, to, tl = attention(p, "tree", mask)
    close(out, want, to)
    close(lse, z, tl)
    # a token's weight was accumulated, then evicted with the weights the GPU holds
    wref, wtol = weight(p, lse, torch.zeros((B, Hkv, S)), 1.0)
    for b in range(B):
        n = min(ctx[b], budget)
        at = token_pos[b, :, :n].long().cpu()
        close(w[b, :, :n], wref[b].gather(1, at), wtol[b].gather(1, at))
        for h in range(Hkv):
            rows = p.cache[p.table[b].long()[at[h] // bs], h, at[h] % bs]
            j = torch.arange(n)
            assert torch.equal(p.d_cache.cpu()[p.table[b].long()[j // bs], h, j % bs].view(torch.uint8), rows.view(torch.uint8))
            if ctx[b] > budget:
                lost = [t for t in range(ctx[b]) if t not in set(at[h].tolist())]
                keep = [t for t in at[h].tolist() if 2 <= t < ctx[b] - 8]
                assert all(2 <= t < ctx[b] - 8 for t in lost)
                assert float(wref[b, h, lost].max()) <= float(wref[b, h, keep].min()) + 2 * float(wtol[b, h].max())
    # attention over the shorter context: request b's first n - 1 places as context, place n - 1 as the drafted token
    s = Problem(1, [min(c, budget) - 1 for c in ctx], (1,) * B, Hq, Hkv, D, bs, fp8)
    s.cache, s.table, s.qkv = p.d_cache.cpu(), p.table, q[:B].cpu()
    want, z, to, tl = attention(s, "dense", None)
    close(out2, want, to)
    close(lse2, z, tl)
    # the same from one captured graph
    p.d_cache.copy_(cache0), w.zero_(), token_pos.copy_(token_pos0)
    first = [x.clone() for x in got]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            again = step()
        for _ in range(2):
            p.d_cache.copy_(cache0), w.zero_(), token_pos.copy_(token_pos0)
            g.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)
