"""Calls of the draft-attention operators at the edges of what their
documentation allows, against the definitions in 64 bits (draft_attn_ref.py)."""

import ctypes
import math
import os

import pytest
import torch

import speculative_decoding_draft_ctx_gb300 as dk
from draft_attn_ref import Problem, attention, close, evict, gen, weight
from test_gpu_draft_attn import cos_sin, kernel, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ a heavy token before a long thin tail


def heavy(n, B, nq, G, Hkv, D, at, gap, fp8=True):
    """B requests over the same n cached tokens: the token at place `at` has V = 0 and a score `gap` nats above all
    others, which are nearly equal and have V around 1, so a row's result is the tail's weights alone."""
    p = Problem(n + D, (n,), (nq,), G * Hkv, Hkv, D, 16, fp8)
    g = gen(n + nq)
    j = torch.arange(n + nq)
    k, v = torch.randn((n + nq, Hkv, D), generator=g) * 0.05, torch.randn((n + nq, Hkv, D), generator=g) * 0.1 + 1.0
    k[at], v[at] = gap / math.sqrt(D), 0.0  # q is about 1 everywhere: q . k / sqrt(D) = gap
    p.write(0, j, k, v)
    p.qkv = (1.0 + 0.05 * torch.randn((B * nq, G * Hkv, D), generator=g)).to(torch.bfloat16)
    p.ctx, p.nq, p.T = [n] * B, [nq] * B, B * nq
    p.start = torch.arange(B + 1, dtype=torch.int32) * nq
    p.table = p.table.repeat(B, 1)
    return p.cuda()


HEAVY = [  # n, requests, nq, G, Hkv, D, place, nats
    (6000, 20, 1, 4, 8, 128, 0, 18.4),  # a CTA has whole items
    (6000, 20, 7, 8, 8, 128, 0, 16.4),
    (6000, 20, 7, 8, 8, 128, 1, 18.4),
    (6000, 10, 20, 8, 8, 128, 0, 18.4),
    (6000, 20, 7, 8, 8, 64, 0, 17.0),
    (6000, 20, 7, 5, 8, 256, 0, 17.0),
    (6000, 20, 7, 8, 8, 128, 5999, 17.0),  # the maximum grows late
    (20000, 1, 7, 8, 4, 128, 0, 17.0),  # items split over CTAs
    (20000, 1, 64, 4, 4, 128, 3000, 18.4),
]


@pytest.mark.parametrize("n,B,nq,G,Hkv,D,at,gap", HEAVY)
def test_attention_tail_behind_a_heavy_token_over_fp8(n, B, nq, G, Hkv, D, at, gap, kernel):  # noqa: F811
    """Weights far below a row's largest keep their bits: every one is at least 2^-28 of the largest, where fp16
    weights with the largest at 2^14 or above are normal numbers, so each is rounded by at most 2^-11 of itself and
    the tolerance of `attention` holds."""
    p = heavy(n, B, nq, G, Hkv, D, at, gap)
    k, _ = p.rows(0)
    for h in range(0, G * Hkv, G):
        x = (p.qkv[:, h].double() @ k[:, h // G].T) * D ** -0.5
        assert 2.0 ** -28 <= (x.amin(1) - x.amax(1)).exp().min() and (x.median(1)[0] - x.amax(1)).exp().max() <= 2.0 ** -22
    out, lse = run_attention(p, "causal", None)
    want, z, to, tl = attention(p, "causal", None)
    close(lse, z, tl)
    close(out, want, to)
    assert int(p.d_flags) == 0


# ------------------------------------------------------------------ eviction: lengths in place


EVICT_LENS = [  # ctx, Hkv, budget, bad lengths in between
    (tuple(300 + i % 40 for i in range(64)), 8, 300, False),  # more (request, head) pairs than CTAs run at once
    ((9000, 30, 8000), 2, 4000, True),  # clusters of several CTAs
    ((50, 60), 3, 80, False),  # nothing to evict: one kernel
]


@pytest.mark.parametrize("ctx,Hkv,budget,bad", EVICT_LENS)
@pytest.mark.parametrize("where", ["context_lens", "seq_lens"])
def test_evict_new_lengths_in_the_place_of_the_old(ctx, Hkv, budget, bad, where):
    """Every head sees the old lengths, and the results are those of a call with lengths of its own."""
    B, S = len(ctx), max(ctx) + 2
    p = Problem(B + Hkv, ctx, (0,) * B, Hkv, Hkv, 64, 16, True).cuda()
    w = torch.rand((B, Hkv, S), generator=gen(3))
    pos = torch.arange(S, dtype=torch.int32).repeat(B, Hkv, 1)
    if bad:
        p.ctx[1] = S + 1
        p.d_ctx[1] = S + 1
    want = evict(p.cache, p.table, 16, [0 if bad and b == 1 else c for b, c in enumerate(p.ctx)], w, pos, ctx, budget, 2, 8)
    want[3][1] = S + 1 if bad else want[3][1]
    for _ in range(3):
        cache, dw, dp = p.d_cache.clone(), w.cuda(), pos.cuda()
        lens, seen = p.d_ctx.clone(), torch.tensor(ctx, dtype=torch.int32, device="cuda")
        new = lens if where == "context_lens" else seen
        assert dk.evict_kv(cache, p.d_table, lens, dw, dp, seen, budget, 2, 8, new_lens=new, error_flags=p.d_flags) is new
        assert new.tolist() == want[3] and int(p.d_flags) == (dk.FLAG_LENGTH if bad else 0)
        assert torch.equal(dw.cpu(), want[1]) and torch.equal(dp.cpu(), want[2]) and torch.equal(cache.cpu(), want[0])


# ------------------------------------------------------------------ scales


@pytest.mark.parametrize("scale,q", [(1e-38, 1e-12), (-1e-38, 1e-12), (1e-30, 2.0 ** -120), (3e-39, 1.0)])
@pytest.mark.parametrize("fp8", [False, True])
def test_attention_scores_that_underflow(scale, q, fp8, kernel):  # noqa: F811
    """Scores below fp32's range are zero: every row is the mean of what it sees."""
    p = Problem(13, (70, 300), (3, 40), 8, 2, 128, 16, fp8)
    p.qkv = (p.qkv.double() * q).to(torch.bfloat16)
    p.cuda()
    out, lse = run_attention(p, "causal", None, scale=scale)
    want, z, to, tl = attention(p, "causal", None, scale=scale)
    close(lse, z, tl)
    close(out, want, to)


@pytest.mark.parametrize("sign", [1, -1])
def test_attention_scores_of_any_size_over_fp8(sign, kernel):  # noqa: F811
    """Scores from 2^9 to 2^33 that grow by 0 to 15 from token to token, around the size from which the weights are
    not lifted: fp32 scores that large decide little, but every result stays among the values it is a mean of."""
    n, nq, G, Hkv, D = 3000, 7, 8, 4, 128
    p = Problem(43, (n,), (nq,), G * Hkv, Hkv, D, 16, True)
    p.k_scale, p.v_scale = torch.ones(1), torch.ones(1)
    g = gen(43)
    k, v = torch.zeros((n + nq, Hkv, D)), torch.randint(8, 17, (n + nq, Hkv, D), generator=g) / 8.0
    k[..., 0], k[..., 1] = 8.0, torch.randint(0, 16, (n + nq, Hkv), generator=g).float()
    p.write(0, torch.arange(n + nq), k, v)
    q = torch.zeros((nq, G * Hkv, D))
    q[..., 1] = 1.0
    size = 2.0 ** (6 + torch.arange(nq * G * Hkv).view(nq, -1) % 24)
    q[..., 0] = sign * size
    p.qkv = q.to(torch.bfloat16)
    p.cuda()
    out, lse = run_attention(p, "dense", None, scale=1.0)
    assert ((out >= 1) & (out <= 2)).all()
    # the largest score, at least, and all tokens at it, at most; a score's own roundings: 3 of 2^-24, 3 more of lse
    top = sign * 8.0 * size.double()
    slack = 6 * 2.0 ** -24 * (top.abs() + 16) + 1e-4
    z = lse.double().cpu()
    assert (z >= top - slack).all() and (z <= top + 15 + math.log(n + nq) + slack).all()
    assert int(p.d_flags) == 0


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_attention_a_scale_that_is_not_a_number_shows(which, kernel):  # noqa: F811
    p = Problem(47, (70, 300), (3, 40), 8, 2, 128, 16, True).cuda()
    (p.d_ks if which == "k_scale" else p.d_vs).fill_(math.nan)
    out, lse = run_attention(p, "causal", None)
    assert out.isnan().all() and (which == "v_scale" or lse.isnan().all())


# ------------------------------------------------------------------ streams


def test_every_operator_on_a_stream_that_is_given():
    """By stream and by handle, with the outputs made by the call: the bits of a call on the current stream."""
    p = Problem(17, (400, 90), (5, 30), 8, 2, 128, 16, True).cuda()
    pos, S = torch.arange(35, device="cuda"), 400
    k = torch.randn((35, 2, 128), device="cuda").to(torch.bfloat16)
    seen = torch.tensor([400, 90], dtype=torch.int32, device="cuda")

    def chain(**kw):
        cache = p.d_cache.clone()
        w, at = torch.zeros((2, 2, S), device="cuda"), torch.arange(S, dtype=torch.int32, device="cuda").repeat(2, 2, 1)
        if kw:
            torch.cuda.synchronize()
        table = dk.rope_table(64, 128, **kw)
        q, k2 = dk.rope_kv_insert(p.d_q, k, table, pos, 128, **kw)
        out, lse = dk.tree_attention(q, cache, p.d_table, p.d_start, p.d_ctx, causal=True, **p.scale_kw(), **kw)
        dk.accumulate_attention_weight(q, cache, p.d_table, p.d_start, p.d_ctx, lse, w, k_scale=p.d_ks, **kw)
        lens = dk.evict_kv(cache, p.d_table, p.d_ctx, w, at, seen, 100, 2, 4, **kw)
        torch.cuda.synchronize()
        return table, q, k2, out, lse, w, at, lens, cache

    want = chain()
    s = torch.cuda.Stream()
    for kw in (dict(stream=s), dict(stream=s.cuda_stream), dict(stream=0)):
        before = torch.cuda.current_stream()
        for a, b in zip(want, chain(**kw)):
            assert torch.equal(a, b)
        assert torch.cuda.current_stream() == before


# ------------------------------------------------------------------ the accumulated weight


@pytest.mark.parametrize("fp8", [False, True])
def test_weight_of_tokens_in_blocks_out_of_range_decays(fp8):
    """With drafted tokens (one group of rows and two) and without."""
    ctx, nq = (100, 100, 300, 40), (3, 0, 40, 2)
    p = Problem(19, ctx, nq, 16, 2, 128, 16, fp8).cuda()
    _, lse = run_attention(p, "dense", None)
    before = torch.rand((4, 2, 305), generator=gen(4))
    good = before.cuda()
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, good, decay=0.5, k_scale=p.d_ks, error_flags=p.d_flags)
    assert int(p.d_flags) == 0
    for b, entry in ((0, -1), (1, 10 ** 6), (2, p.blocks)):
        p.d_table[b, 2] = entry  # tokens 32..47
    got = before.cuda()
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, got, decay=0.5, k_scale=p.d_ks, error_flags=p.d_flags)
    assert int(p.d_flags) == dk.FLAG_BLOCK_RANGE
    want = good.clone()
    want[:3, :, 32:48] = before[:3, :, 32:48].cuda() * 0.5
    assert torch.equal(got, want)


@pytest.mark.parametrize("D,fp8", [(64, False), (128, True), (128, False), (256, True)])
def test_weight_ignores_rows_without_lse_whatever_they_hold(D, fp8):
    """Rows marked as having seen nothing (lse -inf) may hold NaN and infinities; one request has no other rows."""
    ctx, nq = (300, 70, 40), (7, 3, 20)
    p = Problem(23, ctx, nq, 16, 1, D, 16, fp8).cuda()
    _, lse = run_attention(p, "dense", None)
    gone = [2, 5, 7, 8, 9, 29]
    lse[gone] = -math.inf
    w = torch.rand((3, 1, 305), generator=gen(5))
    want = weight(p, lse, w, 0.5)
    blk, off = int(p.table[1, 1]), 3  # token 19 of the request without other rows
    p.d_cache[blk, 0, off, :D] = 0x7F if fp8 else math.nan
    p.d_q[gone] = torch.tensor([math.nan, math.inf, -math.inf, 3e38], dtype=torch.bfloat16, device="cuda").repeat(D // 4)
    got = w.cuda()
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, got, decay=0.5, k_scale=p.d_ks, error_flags=p.d_flags)
    close(got, *want)
    assert int(p.d_flags) == 0


# ------------------------------------------------------------------ waits that run out


@pytest.mark.parametrize("D,fp8", [(64, False), (64, True), (128, False), (128, True)])
def test_expired_waits_report_timeout_and_leave_the_context_usable(D, fp8, monkeypatch):
    """With the test hook the tensor-core kernels' producers copy nothing, so that every role's wait runs out after
    2 ms: the call ends, says so, and the next one is right.  Items of one and of two row tiles, whole and split."""
    p = Problem(29, (900, 3, 400, 3000), (7, 5, 30, 40), 16, 2, D, 16, fp8).cuda()
    monkeypatch.setenv("DSPARK_TREE_ATTN_KERNEL", "tc")
    monkeypatch.setenv("DSPARK_TEST_HOLD_NS", "2000000")
    run_attention(p, "causal", None)
    assert int(p.d_flags) == dk.FLAG_TIMEOUT
    monkeypatch.delenv("DSPARK_TEST_HOLD_NS")
    p.d_flags.zero_()
    out, lse = run_attention(p, "causal", None)
    want, z, to, tl = attention(p, "causal", None)
    close(lse, z, tl)
    close(out, want, to)
    assert int(p.d_flags) == 0
    before = torch.rand((4, 2, 3000), generator=gen(6))
    w = before.cuda()
    kw = dict(decay=0.5, k_scale=p.d_ks, error_flags=p.d_flags)
    monkeypatch.setenv("DSPARK_TEST_HOLD_NS", "2000000")
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, w, **kw)
    assert int(p.d_flags) == dk.FLAG_TIMEOUT
    monkeypatch.delenv("DSPARK_TEST_HOLD_NS")
    p.d_flags.zero_()
    w = before.cuda()
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, w, **kw)
    close(w, *weight(p, lse, before, 0.5))
    assert int(p.d_flags) == 0


def test_expired_waits_of_the_weight_kernel_at_head_dim_256(monkeypatch):
    p = Problem(31, (300, 70), (7, 20), 16, 2, 256, 16, True).cuda()
    _, lse = run_attention(p, "causal", None)
    w = torch.zeros((2, 2, 300), device="cuda")
    monkeypatch.setenv("DSPARK_TEST_HOLD_NS", "2000000")
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, w, k_scale=p.d_ks, error_flags=p.d_flags)
    assert int(p.d_flags) == dk.FLAG_TIMEOUT
    monkeypatch.delenv("DSPARK_TEST_HOLD_NS")
    p.d_flags.zero_(), w.zero_()
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, w, k_scale=p.d_ks, error_flags=p.d_flags)
    close(w, *weight(p, lse, torch.zeros((2, 2, 300)), 1.0))
    assert int(p.d_flags) == 0


# ------------------------------------------------------------------ how kernels follow one another


def programmatic_edges(f):
    """(all edges, those that let a kernel start while the one before drains) of the graph captured from f."""
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        f()
    get = ctypes.CDLL("libcudart.so.13").cudaGraphGetEdges
    get.argtypes, get.restype = [ctypes.c_void_p] * 5, ctypes.c_int
    n = ctypes.c_size_t(0)
    assert get(g.raw_cuda_graph(), None, None, None, ctypes.addressof(n)) == 0
    a, b, data = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (ctypes.c_ubyte * (8 * n.value))()
    assert get(g.raw_cuda_graph(), a, b, data, ctypes.addressof(n)) == 0
    return n.value, sum(data[8 * i + 2] == 1 for i in range(n.value))  # from port, to port, type (1: programmatic), reserved


def test_every_launch_follows_the_switch_for_programmatic_overlap(kernel, monkeypatch):  # noqa: F811
    p = Problem(37, (600, 40), (7, 5), 16, 2, 128, 16, False).cuda()
    out, lse = run_attention(p, "dense", None)
    w, at = torch.rand((2, 2, 600), device="cuda"), torch.arange(600, dtype=torch.int32, device="cuda").repeat(2, 2, 1)
    cos_sin, pos = dk.rope_table(16, 64), torch.arange(12, device="cuda")
    wo, po, lens = torch.empty_like(w), torch.empty_like(at), torch.empty_like(p.d_ctx)

    def chain():
        dk.rope_table(16, 64, out=cos_sin)
        dk.rope_kv_insert(p.d_q, p.d_q[:, :2], cos_sin, pos, 64)
        run_attention(p, "dense", None, out=out, lse=lse)
        dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, w)
        dk.evict_kv(p.d_cache, p.d_table, p.d_ctx, w, at, p.d_ctx, 64, weights_out=wo, positions_out=po, new_lens=lens)

    chain()
    torch.cuda.synchronize()
    edges, overlapped = programmatic_edges(chain)  # table, rotation, attention, join, weight, ranking, moves
    assert edges == 6 and overlapped == 6
    monkeypatch.setenv("DSPARK_PDL", "0")
    assert programmatic_edges(chain) == (6, 0)


# ------------------------------------------------------------------ the kernel that the sizes choose


@pytest.mark.parametrize("fp8", [False, True])
def test_a_batch_of_requests_runs_on_the_tensor_core_kernel(fp8):
    """56 query rows a KV head: without a pin the call has the bits of the tcgen05 kernel, and they are right; so are
    the weights over them."""
    p = Problem(41, (1500, 900, 200, 1300), (7, 7, 7, 7), 16, 2, 128, 16, fp8).cuda()
    out, lse = run_attention(p, "causal", None)
    want, z, to, tl = attention(p, "causal", None)
    close(lse, z, tl)
    close(out, want, to)
    w = torch.zeros((4, 2, 1500), device="cuda")
    dk.accumulate_attention_weight(p.d_q, p.d_cache, p.d_table, p.d_start, p.d_ctx, lse, w, k_scale=p.d_ks, error_flags=p.d_flags)
    close(w, *weight(p, lse, torch.zeros((4, 2, 1500)), 1.0))
    before = os.environ.get("DSPARK_TREE_ATTN_KERNEL")
    os.environ["DSPARK_TREE_ATTN_KERNEL"] = "tc"
    try:
        again = run_attention(p, "causal", None)
    finally:
        os.environ.pop("DSPARK_TREE_ATTN_KERNEL")
        if before is not None:
            os.environ["DSPARK_TREE_ATTN_KERNEL"] = before
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and int(p.d_flags) == 0


# ------------------------------------------------------------------ the table


@pytest.mark.parametrize("theta", [1.5, 1e4])
def test_table_at_the_farthest_positions(theta):
    """The fixed-point turns are off by 2^-64 of a turn (2^-63 with the last one's rounding), 2^-29 radians at 2^31.
    In units of 2^-24: the reduced angle x by 2.47 x (two roundings, and 0.47 of the constant's), which moves an entry
    by x sin x or x cos x of that, 1.37 at pi/4; the last rounding 0.5; of a cosine x^2's 0.25, the series' 0.2 and
    the terms left out 0.42, of a sine 0.2 in all: 2.8."""
    first, r = (1 << 31) - 24, 512
    got = dk.rope_table(24, r, theta=theta, first_position=first, dtype=torch.float32).double().cpu()
    f, _ = dk.rope_frequencies(r, theta)
    want = torch.tensor([[cos_sin(first + p, x) for x in f] for p in range(24)], dtype=torch.float64)
    off = (got.view(24, 2, r // 2) - want.transpose(1, 2)).abs()
    assert off.max() <= 2.8 * 2.0 ** -24 + 2.0 ** -29, float(off.max()) * 2 ** 24
