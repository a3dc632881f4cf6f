"""Refusals and host arithmetic of the draft-attention operators at the edges
of what their documentation allows.  No test here launches a kernel."""

import math
import types

import pytest
import torch

import speculative_decoding_draft_ctx_gb300 as dk
from speculative_decoding_draft_ctx_gb300 import draft_attn
from test_draft_attn_cpu import EVICT, EVICT_BASE, FAKE, L, args, refuses, status, table_call  # noqa: F401

# arrays of their own, 64 KB apart: every call below is refused before any CUDA call
APART = {**EVICT_BASE, **{k: FAKE * (2 + i) for i, k in enumerate("ctx w pos wo po seen lens".split())}}


@pytest.mark.parametrize("over", [
    dict(lens=APART["ctx"] + 4), dict(lens=APART["ctx"] - 4), dict(lens=APART["seen"] + 4), dict(ctx=APART["lens"] + 4)])
def test_evict_refuses_lengths_that_overlap_partly(L, over):  # noqa: F811
    assert status(L, "dspark_kv_evict", EVICT, APART, over) == "DSPARK_ERR_INVALID_ARG"
    assert "new_lens" in dk.dspark_ctx_kv_last_error()


@pytest.mark.parametrize("over", [
    dict(wo=APART["w"] + 4), dict(wo=APART["w"] - 1020), dict(po=APART["pos"] + 1020), dict(w=APART["wo"] + 4), dict(wo=APART["pos"]),
    dict(po=APART["w"]), dict(wo=APART["po"]), dict(wo=APART["po"] + 4), dict(po=APART["w"] + 8)])
def test_evict_refuses_outputs_that_overlap_partly(L, over):  # noqa: F811
    """2 requests x 2 heads x 64 places of 4 bytes: 1,024 bytes each."""
    assert status(L, "dspark_kv_evict", EVICT, APART, over) == "DSPARK_ERR_INVALID_ARG"
    assert "overlap" in dk.dspark_ctx_kv_last_error()


def test_a_stream_of_another_device_is_refused():
    draft_attn._load()
    here, there = torch.device("cuda", 0), torch.device("cuda", 1)
    with pytest.raises(dk.DSparkError, match="stream is on cuda:1"):
        draft_attn._elsewhere(here, types.SimpleNamespace(device=there, cuda_stream=FAKE))
    assert draft_attn._elsewhere(there, types.SimpleNamespace(device=there, cuda_stream=FAKE))
    assert draft_attn._elsewhere(here, FAKE)  # a handle says nothing about its device


@pytest.mark.parametrize("r", [2, 6, 64, 128])
@pytest.mark.parametrize("theta", [1.5, 1e4, 1e6])
@pytest.mark.parametrize("L,fast,slow", [(4096, 32, 1), (64, 32, 16), (64, 32, 11), (6, 32, 1), (1, 32, 1), (1, 0.5, 0.1), (2 ** 20, 32, 1), (100, 8, 7.9)])
def test_by_parts_keeps_and_divides_what_it_says(r, theta, L, fast, slow):
    """Dims that turn at least beta_fast times in L keep their frequency, those that turn at most beta_slow times are
    divided, the others lie between, falling."""
    base, _ = dk.rope_frequencies(r, theta)
    got, _ = dk.rope_frequencies(r, theta, dict(kind="by_parts", factor=8, original_positions=L, beta_fast=fast, beta_slow=slow))
    shares = [(y / x - 1 / 8) / (1 - 1 / 8) for x, y in zip(base, got)]
    for f, share in zip(base, shares):
        turns = f * L / (2 * math.pi)
        assert -1e-12 <= share <= 1 + 1e-12
        if turns >= fast * (1 + 1e-9):
            assert abs(share - 1) < 1e-12
        if turns <= slow * (1 - 1e-9):
            assert abs(share) < 1e-12
    assert all(a >= b - 1e-12 for a, b in zip(shares, shares[1:]))


def test_by_parts_refuses_betas_without_end():
    with pytest.raises(dk.DSparkError, match="beta_fast"):
        dk.rope_frequencies(64, 1e4, dict(kind="by_parts", factor=8, original_positions=64, beta_fast=math.inf))


# ------------------------------------------------------------------ numbers that the C types do not hold


@pytest.mark.parametrize("kw", [dict(first_position=1 << 64), dict(first_position=(1 << 31) + 1), dict(first_position=-1), dict(num_positions=1 << 64),
                                dict(num_positions=(1 << 31) - 9, first_position=10)])
def test_table_refuses_positions_beyond_its_range(kw):
    with pytest.raises(dk.DSparkError, match="2.31"):
        dk.rope_table(**{**dict(num_positions=4, rotary_dim=16, device="cpu"), **kw})


@pytest.mark.parametrize("amp", [1e39, -1e300])
def test_table_refuses_an_amplitude_beyond_fp32(L, amp):  # noqa: F811
    assert table_call(L, amp=amp) == "DSPARK_ERR_INVALID_ARG"


@pytest.mark.parametrize("kw,match", [(dict(budget=1 << 64), "expected a CUDA device"), (dict(budget=(1 << 64) + 5, sinks=9), "expected a CUDA device"),
                                      (dict(budget=5, sinks=1 << 64), "budget"), (dict(budget=1 << 64, recent=1 << 64), "expected a CUDA device"), (dict(budget=-1 << 64), "budget")])
def test_evict_takes_budgets_beyond_64_bits_for_what_they_are(kw, match):
    """A budget above every length: the call is refused for its CPU tensors alone; counts above the budget are not."""
    a = args()
    base = dict(kv_cache=a["kv_cache"], block_table=a["block_table"], context_lens=a["context_lens"], weights=torch.zeros((2, 2, 9)),
                token_positions=torch.zeros((2, 2, 9), dtype=torch.int32), seq_lens=torch.zeros(2, dtype=torch.int32))
    refuses(dk.evict_kv, **{**base, **kw}, match=match)


def test_workspace_queries_refuse_the_sizes_that_the_calls_refuse(L):  # noqa: F811
    big = 2 ** 31 - 1
    for a in ((big, big, 100, 60), (1 << 27, 1, 100, 60), (1, 1, big, 60), (1, 1, 1 << 62, 1 << 61), (-1, 1, 9, 9), (1, 0, 9, 9), (1, 1, -1, 9)):
        assert L.dspark_kv_evict_workspace(*a) == -1, a
    assert L.dspark_kv_evict_workspace((1 << 27) - 1, 1, 1 << 30, 1 << 29) == ((1 << 27) - 1) * (1 + (1 << 30)) * 4
    assert L.dspark_kv_evict_workspace(2, 3, 9, 1 << 62) == 24
    for a in ((1 << 62, 8, 1, 128, 4, 0), (1 << 29, 8, 1, 128, 4, 0), (5, 1 << 21, 1, 128, 4, 0), (5, 1 << 17, 1 << 17, 128, 4, 0), (5, 8, 2, 128, 1 << 25, 0),
              (-1, 8, 2, 128, 4, 0), (5, 8, 2, 128, -1, 0)):
        assert L.dspark_tree_attention_workspace(*a) == -1, a
