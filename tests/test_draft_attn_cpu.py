"""The draft-attention operators without a GPU: every precondition becomes its
status before any CUDA call, sizes of zero launch nothing, the Python layer
refuses what does not fit, and the scaled frequencies follow their formulas.
No test here launches a kernel."""

import ctypes
import math

import pytest
import torch

import speculative_decoding_draft_ctx_gb300 as dk
from speculative_decoding_draft_ctx_gb300 import build as kbuild

FAKE = 0x10000  # an aligned address that is never dereferenced: every call below fails validation or has nothing to do


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return dk.lib()


def status(L, name, order, base, over):
    a = dict(base)
    assert set(over) <= set(a), set(over) - set(a)
    a.update(over)
    return dk.STATUS[getattr(L, name)(*[a[k] for k in order.split()])]


# ------------------------------------------------------------------ the C boundary

TABLE = "out first count r freqs amp fp32 stream"


def table_call(L, freqs=(1.0,) * 8, **over):
    base = dict(out=FAKE, first=0, count=4, r=16, freqs=freqs and (ctypes.c_double * len(freqs))(*freqs), amp=1.0, fp32=0, stream=0)
    return status(L, "dspark_rope_table", TABLE, base, over)


@pytest.mark.parametrize("over,want", [
    (dict(r=0), "DSPARK_ERR_UNSUPPORTED_ROTARY_DIM"), (dict(r=7), "DSPARK_ERR_UNSUPPORTED_ROTARY_DIM"),
    (dict(r=514), "DSPARK_ERR_UNSUPPORTED_ROTARY_DIM"), (dict(first=-1), "DSPARK_ERR_INVALID_ARG"),
    (dict(count=-1), "DSPARK_ERR_INVALID_ARG"), (dict(first=(1 << 31) - 3), "DSPARK_ERR_INVALID_ARG"),
    (dict(amp=math.nan), "DSPARK_ERR_INVALID_ARG"), (dict(freqs=None), "DSPARK_ERR_INVALID_ARG"),
    (dict(out=0), "DSPARK_ERR_INVALID_ARG"), (dict(out=FAKE + 4), "DSPARK_ERR_ALIGNMENT"), (dict(count=0), "DSPARK_OK")])
def test_table_status(L, over, want):
    assert table_call(L, **over) == want


def test_table_refuses_a_frequency_that_is_not_finite(L):
    assert table_call(L, freqs=(1.0,) * 7 + (math.inf,)) == "DSPARK_ERR_INVALID_ARG"
    assert "freqs[7]" in dk.dspark_ctx_kv_last_error()


ROPE = ("q qts qhs k kts khs v vts vhs qo qots qohs ko kots kohs cs fp32 max_pos pos T Hq Hkv D r inter inv slots cache blocks bs dt ks vs "
        "flags stream")
ROPE_BASE = dict(q=FAKE, qts=512, qhs=128, k=FAKE, kts=512, khs=128, v=FAKE, vts=512, vhs=128, qo=FAKE, qots=512, qohs=128, ko=FAKE, kots=512,
                 kohs=128, cs=FAKE, fp32=0, max_pos=64, pos=FAKE, T=4, Hq=2, Hkv=1, D=128, r=64, inter=0, inv=0, slots=FAKE, cache=FAKE,
                 blocks=4, bs=16, dt=0, ks=0, vs=0, flags=0, stream=0)


@pytest.mark.parametrize("over,want", [
    (dict(D=96), "DSPARK_ERR_INVALID_ARG"), (dict(r=3), "DSPARK_ERR_UNSUPPORTED_ROTARY_DIM"), (dict(r=130), "DSPARK_ERR_UNSUPPORTED_ROTARY_DIM"),
    (dict(r=0), "DSPARK_ERR_UNSUPPORTED_ROTARY_DIM"), (dict(Hq=0), "DSPARK_ERR_INVALID_ARG"), (dict(Hkv=0), "DSPARK_ERR_INVALID_ARG"),
    (dict(T=-1), "DSPARK_ERR_INVALID_ARG"), (dict(max_pos=0), "DSPARK_ERR_INVALID_ARG"), (dict(slots=0), "DSPARK_ERR_INVALID_ARG"),
    (dict(cache=0), "DSPARK_ERR_INVALID_ARG"), (dict(v=0), "DSPARK_ERR_INVALID_ARG"), (dict(bs=0), "DSPARK_ERR_BLOCK_SIZE"),
    (dict(dt=5), "DSPARK_ERR_DTYPE"), (dict(blocks=0), "DSPARK_ERR_INVALID_ARG"), (dict(blocks=1 << 60), "DSPARK_ERR_INVALID_ARG"),
    (dict(cache=FAKE + 8), "DSPARK_ERR_ALIGNMENT"), (dict(q=FAKE + 1), "DSPARK_ERR_ALIGNMENT"), (dict(cs=FAKE + 8), "DSPARK_ERR_ALIGNMENT"),
    (dict(pos=FAKE + 4), "DSPARK_ERR_ALIGNMENT"), (dict(slots=FAKE + 4), "DSPARK_ERR_ALIGNMENT"), (dict(ks=FAKE + 2), "DSPARK_ERR_ALIGNMENT"),
    (dict(qts=1 << 41), "DSPARK_ERR_INVALID_ARG"), (dict(q=0), "DSPARK_ERR_INVALID_ARG"), (dict(T=0), "DSPARK_OK"),
    (dict(T=0, slots=0, cache=0, v=0), "DSPARK_OK")])
def test_rope_status(L, over, want):
    assert status(L, "dspark_rope_kv_insert", ROPE, ROPE_BASE, over) == want


ATTN = ("q qts qhs T Hq Hkv D cache blocks bs dt ks vs table ts tb start ctx B kind mask words scale out lse ws wsb flags stream")
ATTN_BASE = dict(q=FAKE, qts=1024, qhs=128, T=4, Hq=8, Hkv=2, D=128, cache=FAKE, blocks=8, bs=16, dt=0, ks=0, vs=0, table=FAKE, ts=4, tb=4,
                 start=FAKE, ctx=FAKE, B=2, kind=0, mask=0, words=0, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 30, flags=0, stream=0)
QUERY_RULES = [
    (dict(D=32), "DSPARK_ERR_INVALID_ARG"), (dict(Hkv=0), "DSPARK_ERR_INVALID_ARG"), (dict(Hq=7), "DSPARK_ERR_INVALID_ARG"),
    (dict(Hq=0), "DSPARK_ERR_INVALID_ARG"), (dict(T=-1), "DSPARK_ERR_INVALID_ARG"), (dict(T=1 << 31), "DSPARK_ERR_INVALID_ARG"),
    (dict(blocks=0), "DSPARK_ERR_INVALID_ARG"), (dict(bs=0), "DSPARK_ERR_BLOCK_SIZE"), (dict(dt=2), "DSPARK_ERR_DTYPE"),
    (dict(cache=0), "DSPARK_ERR_INVALID_ARG"), (dict(cache=FAKE + 4), "DSPARK_ERR_ALIGNMENT"), (dict(q=FAKE + 8), "DSPARK_ERR_ALIGNMENT"),
    (dict(qts=1028), "DSPARK_ERR_ALIGNMENT"), (dict(qhs=132), "DSPARK_ERR_ALIGNMENT"), (dict(ts=3), "DSPARK_ERR_INVALID_ARG"),
    (dict(tb=0), "DSPARK_ERR_INVALID_ARG"), (dict(table=0), "DSPARK_ERR_INVALID_ARG"), (dict(table=FAKE + 2), "DSPARK_ERR_ALIGNMENT"),
    (dict(B=-1), "DSPARK_ERR_INVALID_ARG"), (dict(scale=math.inf), "DSPARK_ERR_INVALID_ARG"), (dict(scale=math.nan), "DSPARK_ERR_INVALID_ARG"),
    (dict(start=0), "DSPARK_ERR_INVALID_ARG"), (dict(q=0), "DSPARK_ERR_INVALID_ARG"), (dict(ks=FAKE + 1), "DSPARK_ERR_ALIGNMENT"),
    (dict(flags=FAKE + 1), "DSPARK_ERR_ALIGNMENT")]


@pytest.mark.parametrize("over,want", QUERY_RULES + [
    (dict(kind=3), "DSPARK_ERR_INVALID_ARG"), (dict(kind=2, words=0, mask=FAKE), "DSPARK_ERR_INVALID_ARG"),
    (dict(kind=2, words=1, mask=0), "DSPARK_ERR_INVALID_ARG"), (dict(kind=2, words=1, mask=FAKE + 4), "DSPARK_ERR_ALIGNMENT"),
    (dict(out=0), "DSPARK_ERR_INVALID_ARG"), (dict(out=FAKE + 2), "DSPARK_ERR_ALIGNMENT"), (dict(lse=0), "DSPARK_ERR_INVALID_ARG"),
    (dict(ws=FAKE + 8), "DSPARK_ERR_ALIGNMENT"), (dict(T=0), "DSPARK_OK"), (dict(B=0), "DSPARK_OK")])
def test_attention_status(L, over, want):
    assert status(L, "dspark_tree_attention", ATTN, ATTN_BASE, over) == want


WEIGHT = "q qts qhs T Hq Hkv D cache blocks bs dt ks table ts tb start ctx B lse scale decay w places flags stream"
WEIGHT_BASE = {**{k: ATTN_BASE[k] for k in WEIGHT.split() if k in ATTN_BASE}, "decay": 0.9, "w": FAKE, "places": 64}


@pytest.mark.parametrize("over,want", QUERY_RULES + [
    (dict(decay=math.nan), "DSPARK_ERR_INVALID_ARG"), (dict(places=-1), "DSPARK_ERR_INVALID_ARG"), (dict(w=0), "DSPARK_ERR_INVALID_ARG"),
    (dict(w=FAKE + 2), "DSPARK_ERR_ALIGNMENT"), (dict(lse=0), "DSPARK_ERR_INVALID_ARG"), (dict(places=0), "DSPARK_OK"), (dict(B=0), "DSPARK_OK")])
def test_weight_status(L, over, want):
    assert status(L, "dspark_attention_weight_accumulate", WEIGHT, WEIGHT_BASE, over) == want


EVICT = "cache blocks Hkv bs D dt table ts tb ctx B w pos wo po places seen budget sinks recent lens ws wsb flags stream"
EVICT_BASE = dict(cache=FAKE, blocks=8, Hkv=2, bs=16, D=128, dt=0, table=FAKE, ts=4, tb=4, ctx=FAKE, B=2, w=FAKE, pos=FAKE, wo=FAKE, po=FAKE,
                  places=64, seen=FAKE, budget=32, sinks=4, recent=8, lens=FAKE, ws=FAKE, wsb=1 << 20, flags=0, stream=0)


@pytest.mark.parametrize("over,want", [
    (dict(D=100), "DSPARK_ERR_INVALID_ARG"), (dict(bs=-1), "DSPARK_ERR_BLOCK_SIZE"), (dict(dt=9), "DSPARK_ERR_DTYPE"),
    (dict(cache=0), "DSPARK_ERR_INVALID_ARG"), (dict(cache=FAKE + 1), "DSPARK_ERR_ALIGNMENT"), (dict(budget=0), "DSPARK_ERR_INVALID_ARG"),
    (dict(sinks=-1), "DSPARK_ERR_INVALID_ARG"), (dict(recent=-1), "DSPARK_ERR_INVALID_ARG"), (dict(sinks=25), "DSPARK_ERR_INVALID_ARG"),
    (dict(sinks=1 << 62, recent=1 << 62), "DSPARK_ERR_INVALID_ARG"), (dict(places=-1), "DSPARK_ERR_INVALID_ARG"),
    (dict(places=1 << 31), "DSPARK_ERR_INVALID_ARG"), (dict(w=0), "DSPARK_ERR_INVALID_ARG"), (dict(lens=0), "DSPARK_ERR_INVALID_ARG"),
    (dict(seen=0), "DSPARK_ERR_INVALID_ARG"), (dict(pos=FAKE + 2), "DSPARK_ERR_ALIGNMENT"), (dict(wsb=100), "DSPARK_ERR_INVALID_ARG"),
    (dict(ws=0), "DSPARK_ERR_INVALID_ARG"), (dict(ws=FAKE + 4), "DSPARK_ERR_ALIGNMENT"), (dict(tb=0), "DSPARK_ERR_INVALID_ARG"),
    (dict(B=0), "DSPARK_OK")])
def test_evict_status(L, over, want):
    assert status(L, "dspark_kv_evict", EVICT, EVICT_BASE, over) == want


def test_workspaces(L):
    # a count and two lists of at most min(budget, places - budget) entries of 4 bytes per request and head
    assert L.dspark_kv_evict_workspace(3, 2, 100, 60) == 3 * 2 * (1 + 2 * 40) * 4
    assert L.dspark_kv_evict_workspace(3, 2, 100, 100) == 24 and L.dspark_kv_evict_workspace(3, 2, 10, 100) == 24
    assert L.dspark_kv_evict_workspace(3, 2, 100, 0) == -1
    assert L.dspark_tree_attention_workspace(0, 8, 2, 128, 4, 0) == 0 and L.dspark_tree_attention_workspace(5, 8, 2, 128, 0, 0) == 0
    assert L.dspark_tree_attention_workspace(5, 8, 3, 128, 4, 0) == -1 and L.dspark_tree_attention_workspace(5, 8, 2, 80, 4, 0) == -1


# ------------------------------------------------------------------ the Python layer


def refuses(f, *a, match=None, **kw):
    with pytest.raises(dk.DSparkError, match=match) as e:
        f(*a, **kw)
    assert e.value.status in (1, 2)


def args(T=4, Hq=4, Hkv=2, D=64, B=2, fp8=False):
    return dict(q=torch.zeros((T, Hq, D), dtype=torch.bfloat16),
                kv_cache=torch.zeros((3, Hkv, 16, 2 * D), dtype=torch.uint8 if fp8 else torch.bfloat16),
                block_table=torch.zeros((B, 2), dtype=torch.int32), query_start=torch.zeros(B + 1, dtype=torch.int32),
                context_lens=torch.zeros(B, dtype=torch.int32))


@pytest.mark.parametrize("over,match", [
    (dict(q=torch.zeros((4, 4, 64))), "bfloat16"), (dict(q=torch.zeros((4, 256), dtype=torch.bfloat16)), "3 dims"),
    (dict(q=torch.zeros((4, 4, 128), dtype=torch.bfloat16)), "do not match"), (dict(q=torch.zeros((4, 3, 64), dtype=torch.bfloat16)), "do not match"),
    (dict(q=torch.zeros((4, 64, 4), dtype=torch.bfloat16).transpose(1, 2)), "head rows"),
    (dict(kv_cache=torch.zeros((3, 2, 16, 96), dtype=torch.bfloat16)), "rows hold"), (dict(kv_cache=torch.zeros((3, 2, 16, 128))), "kv_cache"),
    (dict(kv_cache=torch.zeros((3, 16, 2, 128), dtype=torch.bfloat16).transpose(1, 2)), "contiguous"),
    (dict(block_table=torch.zeros((2, 2), dtype=torch.int64)), "block_table"), (dict(block_table=torch.zeros((2, 0), dtype=torch.int32)), "block_table"),
    (dict(block_table=torch.zeros((2, 4), dtype=torch.int32)[:, ::2]), "block_table"),
    (dict(query_start=torch.zeros(2, dtype=torch.int32)), "query_start"), (dict(query_start=torch.zeros(3, dtype=torch.int64)), "query_start"),
    (dict(context_lens=torch.zeros(3, dtype=torch.int32)), "context_lens"), (dict(tree_mask=torch.zeros((4, 1))), "tree_mask"),
    (dict(tree_mask=torch.zeros((3, 1), dtype=torch.int64)), "tree_mask"), (dict(tree_mask=torch.zeros((4, 0), dtype=torch.int64)), "tree_mask"),
    (dict(tree_mask=torch.zeros((4, 1), dtype=torch.int64), causal=True), "exclude"), (dict(out=torch.zeros((4, 4, 64))), "out"),
    (dict(lse=torch.zeros((4, 2))), "lse"), (dict(k_scale=torch.zeros(1, dtype=torch.bfloat16)), "k_scale"),
    (dict(error_flags=torch.zeros(1)), "error_flags"), (dict(), "expected a CUDA device")])
def test_attention_refuses(over, match):
    refuses(dk.tree_attention, **{**args(), **over}, match=match)


@pytest.mark.parametrize("over,match", [
    (dict(lse=torch.zeros((4, 2))), "lse"), (dict(weights=torch.zeros((2, 3, 9))), "weights"), (dict(weights=torch.zeros((3, 2, 9))), "weights"),
    (dict(weights=torch.zeros((2, 2, 9)).double()), "weights"), (dict(), "expected a CUDA device")])
def test_weight_refuses(over, match):
    refuses(dk.accumulate_attention_weight, **{**args(), "lse": torch.zeros((4, 4)), "weights": torch.zeros((2, 2, 9)), **over}, match=match)


@pytest.mark.parametrize("over,match", [
    (dict(weights=torch.zeros((2, 1, 9))), "weights"), (dict(token_positions=torch.zeros((2, 2, 8), dtype=torch.int32)), "token_positions"),
    (dict(token_positions=torch.zeros((2, 2, 9))), "token_positions"), (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), "seq_lens"),
    (dict(weights_out=torch.zeros((2, 2, 8))), "weights_out"), (dict(positions_out=torch.zeros((2, 2, 9))), "positions_out"),
    (dict(new_lens=torch.zeros(1, dtype=torch.int32)), "new_lens"), (dict(budget=0), "budget"), (dict(sinks=3, recent=3), "budget"),
    (dict(), "expected a CUDA device")])
def test_evict_refuses(over, match):
    a = args()
    base = dict(kv_cache=a["kv_cache"], block_table=a["block_table"], context_lens=a["context_lens"], weights=torch.zeros((2, 2, 9)),
                token_positions=torch.zeros((2, 2, 9), dtype=torch.int32), seq_lens=torch.zeros(2, dtype=torch.int32), budget=5)
    refuses(dk.evict_kv, **{**base, **over}, match=match)


@pytest.mark.parametrize("over,match", [
    (dict(layout="neox"), "layout"), (dict(rotary_dim=16), "rotary_dim"), (dict(cos_sin_cache=torch.zeros((8, 32)).double()), "cos_sin_cache"),
    (dict(positions=torch.zeros(3, dtype=torch.int64)), "positions"), (dict(positions=torch.zeros(4, dtype=torch.int32)), "positions"),
    (dict(k=torch.zeros((3, 2, 64), dtype=torch.bfloat16)), "k has shape"), (dict(slot_mapping=torch.zeros(4, dtype=torch.int64)), "go together"),
    (dict(slot_mapping=torch.zeros(4, dtype=torch.int64), kv_cache=args()["kv_cache"]), "go together"),
    (dict(slot_mapping=torch.zeros(2, dtype=torch.int64), kv_cache=args()["kv_cache"], v=torch.zeros((4, 2, 64), dtype=torch.bfloat16)), "slot_mapping"),
    (dict(slot_mapping=torch.zeros(4, dtype=torch.int64), kv_cache=args(Hkv=1)["kv_cache"], v=torch.zeros((4, 2, 64), dtype=torch.bfloat16)), "kv_cache"),
    (dict(q_out=torch.zeros((4, 2, 64), dtype=torch.bfloat16)), "q_out"), (dict(), "expected a CUDA device")])
def test_rope_refuses(over, match):
    base = dict(q=torch.zeros((4, 4, 64), dtype=torch.bfloat16), k=torch.zeros((4, 2, 64), dtype=torch.bfloat16), cos_sin_cache=torch.zeros((8, 32)),
                positions=torch.zeros(4, dtype=torch.int64), rotary_dim=32)
    refuses(dk.rope_kv_insert, **{**base, **over}, match=match)


@pytest.mark.parametrize("kw,match", [
    (dict(rotary_dim=5), "rotary_dim"), (dict(theta=1.0), "theta"), (dict(scaling=dict(kind="other", factor=2)), "kind"),
    (dict(scaling=dict(kind="linear")), "factor"), (dict(scaling=dict(kind="linear", factor=0.5)), "factor"),
    (dict(scaling=dict(kind="by_parts", factor=2)), "original_positions"), (dict(scaling=dict(kind="linear", factor=2, beta=1)), "unknown"),
    (dict(scaling=dict(kind="by_parts", factor=2, original_positions=64, beta_fast=1, beta_slow=2)), "beta_fast"),
    (dict(scaling=dict(kind="bands", factor=2, original_positions=64, low_freq_factor=4)), "high_freq_factor"),
    (dict(dtype=torch.float16), "dtype"), (dict(num_positions=-1), "num_positions"), (dict(device="cpu"), "expected a CUDA device"),
    (dict(out=torch.zeros((4, 8))), "out must have shape"), (dict(out=torch.zeros((4, 16)), dtype=torch.bfloat16), "dtype")])
def test_table_refuses(kw, match):
    refuses(dk.rope_table, **{**dict(num_positions=4, rotary_dim=16, device="cpu"), **kw}, match=match)


# ------------------------------------------------------------------ scaled frequencies


def test_frequencies():
    base, amp = dk.rope_frequencies(64, 1e4)
    assert amp == 1.0 and base[0] == 1.0 and abs(base[16] - 0.01) < 1e-15
    lin, _ = dk.rope_frequencies(64, 1e4, dict(kind="linear", factor=8))
    assert all(abs(8 * x - y) <= 1e-15 * y for x, y in zip(lin, base))
    # by parts: whole above beta_fast turns over the original length, divided below beta_slow, monotone between
    L, s = 4096, 4.0
    parts, amp = dk.rope_frequencies(64, 1e4, dict(kind="by_parts", factor=s, original_positions=L))
    assert abs(amp - (0.1 * math.log(s) + 1)) < 1e-15
    turns = [L * x / (2 * math.pi) for x in base]
    share = [(y / x - 1 / s) / (1 - 1 / s) for x, y in zip(base, parts)]
    for i, t in enumerate(turns):
        if t > 32:
            assert abs(share[i] - 1) < 1e-12
        if t < 1:
            assert abs(share[i]) < 0.1 and (i + 1 >= len(turns) or share[i + 1] <= share[i] + 1e-12)
    assert share[0] > 0.999 and abs(share[-1]) < 1e-12 and all(a >= b - 1e-12 for a, b in zip(share, share[1:]))
    # bands: exactly halfway at the middle number of turns
    mid = 2 * math.pi * 2.5 / L
    theta = (1 / mid) ** (64 / 32)  # frequency 16 of 64 turns 2.5 times
    bands, _ = dk.rope_frequencies(64, theta, dict(kind="bands", factor=8, original_positions=L))
    assert abs(bands[16] - (0.5 * mid + 0.5 * mid / 8)) < 1e-9 * mid
    assert bands[0] == 1.0 and abs(bands[31] - dk.rope_frequencies(64, theta)[0][31] / 8) < 1e-18


def test_fixed_point_turns():
    """The integer range reduction of the table, in Python: the fraction of a turn of p f is p F mod 2^64."""
    from fractions import Fraction

    for f in (1.0, 0.25, 1e-4, 3.7e-7):
        turn = f / (2 * math.pi)
        F = int(math.ldexp(turn - math.floor(turn), 64))
        for p in (0, 1, 12345, (1 << 31) - 1):
            u = (p * F) % (1 << 64)
            want = Fraction(turn) * p
            d = abs(Fraction(u, 1 << 64) - (want - math.floor(want)))
            assert min(d, 1 - d) <= Fraction(p + 1, 1 << 64)
            quarter = ((u + (1 << 61)) % (1 << 64)) >> 62
            rest = (u - (quarter << 62)) % (1 << 64)
            rest -= (1 << 64) if rest >= 1 << 63 else 0
            assert -(1 << 61) <= rest < 1 << 61
