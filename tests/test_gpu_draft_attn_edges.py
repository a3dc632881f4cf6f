"""Calls of the draft-attention operators at the edges of what their
documentation allows, against the definitions in 64 bits (draft_attn_ref.py)."""

import math

import pytest
import torch

import speculative_decoding_draft_ctx_gb300 as dk
from draft_attn_ref import Problem, attention, close, gen, tree_mask
from test_gpu_draft_attn import kernel, run_attention  # noqa: F401

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
