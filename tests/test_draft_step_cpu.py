"""The draft-step operators without a GPU: every precondition becomes its status
before any CUDA call, sizes of zero launch nothing, and the Python layer
refuses what does not fit.  No test here launches a kernel."""

import ctypes

import pytest
import torch

import speculative_decoding_draft_ctx_gb300 as dk
from draft_step_ref import Pool, encode, exponent, grow, value, verify
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


def layers(*at):
    return (ctypes.c_void_p * len(at))(*at)


BAD, ALIGN, DTYPE, OK, BLOCK = "DSPARK_ERR_INVALID_ARG", "DSPARK_ERR_ALIGNMENT", "DSPARK_ERR_DTYPE", "DSPARK_OK", "DSPARK_ERR_BLOCK_SIZE"

# ------------------------------------------------------------------ the C boundary

VERIFY = "t tt ts d dt ds rows vocab tok up u start B most repl ot orow oc flags stream"
VERIFY_BASE = dict(t=FAKE, tt=0, ts=100, d=FAKE, dt=1, ds=100, rows=8, vocab=100, tok=FAKE, up=FAKE, u=FAKE, start=FAKE, B=2, most=4, repl=1,
                   ot=FAKE, orow=FAKE, oc=FAKE, flags=0, stream=0)


@pytest.mark.parametrize("over,want", [
    (dict(tt=2), DTYPE), (dict(dt=-1), DTYPE), (dict(vocab=0), BAD), (dict(vocab=(1 << 30) + 1), BAD), (dict(rows=-1), BAD), (dict(B=-1), BAD),
    (dict(most=0), BAD), (dict(most=1024), BAD), (dict(ts=1 << 50), BAD), (dict(t=0), BAD), (dict(tok=0), BAD), (dict(u=0), BAD),
    (dict(start=0), BAD), (dict(ot=0), BAD), (dict(orow=0), BAD), (dict(oc=0), BAD), (dict(t=FAKE + 2), ALIGN), (dict(d=FAKE + 1), ALIGN),
    (dict(tok=FAKE + 4), ALIGN), (dict(ot=FAKE + 4), ALIGN), (dict(up=FAKE + 2), ALIGN), (dict(flags=FAKE + 1), ALIGN), (dict(B=0), OK)])
def test_verify_status(L, over, want):
    assert status(L, "dspark_verify_drafts", VERIFY, VERIFY_BASE, over) == want


VERIFY_APART = dict(VERIFY_BASE, t=FAKE, d=FAKE + 8192, tok=FAKE + 16384, up=FAKE + 16640, u=FAKE + 16896, start=FAKE + 17152, ot=FAKE + 17408,
                    orow=FAKE + 17664, oc=FAKE + 17920)


@pytest.mark.parametrize("over", [
    dict(ot=FAKE + 3192), dict(ot=FAKE + 8192 + 1592), dict(oc=FAKE + 8192 - 4), dict(ot=FAKE + 16384 - 72), dict(ot=FAKE + 16384 + 56),
    dict(orow=FAKE + 16640), dict(oc=FAKE + 16640 + 28), dict(orow=FAKE + 16896 + 28), dict(oc=FAKE + 17152 + 8), dict(ot=FAKE + 17152),
    dict(orow=FAKE + 17408 + 76), dict(oc=FAKE + 17408 + 76), dict(oc=FAKE + 17664 + 28), dict(d=0, t=FAKE + 4096, ts=-100, ot=FAKE + 4096 - 2872),
    dict(ts=0, oc=FAKE + 396), dict(ts=1024, oc=FAKE + 4096 + 396), dict(ts=1 << 40, oc=FAKE + (7 << 42)), dict(ds=-(1 << 40), d=8 << 41, oc=1 << 41)])
def test_verify_refuses_outputs_over_inputs_or_one_another(L, over):
    """The first or last bytes of a buffer or row."""
    assert status(L, "dspark_verify_drafts", VERIFY, VERIFY_APART, over) == BAD
    assert b"overlap" in L.dspark_ctx_kv_last_error()


COMPACT = "caches scales L blocks nkv bs D dt table stride cols ctx B rows rstride width counts first lens flags stream"
COMPACT_BASE = dict(caches=layers(FAKE, FAKE + 4096), scales=None, L=2, blocks=4, nkv=2, bs=16, D=128, dt=0, table=FAKE, stride=4, cols=4, ctx=FAKE, B=3,
                    rows=FAKE + 256, rstride=4, width=4, counts=FAKE + 512, first=1, lens=FAKE + 1024, flags=0, stream=0)


@pytest.mark.parametrize("over,want", [
    (dict(L=0), BAD), (dict(caches=None), BAD), (dict(caches=layers(FAKE, 0)), BAD), (dict(caches=layers(FAKE, FAKE + 8)), ALIGN),
    (dict(scales=layers(FAKE, FAKE + 64)), DTYPE), (dict(caches=layers(FAKE, FAKE)), BAD), (dict(scales=layers(FAKE, FAKE), dt=1), BAD),
    (dict(L=1025), BAD), (dict(scales=layers(FAKE, 0), dt=1), BAD), (dict(D=96), BAD), (dict(bs=0), BLOCK), (dict(dt=7), DTYPE),
    (dict(blocks=0), BAD), (dict(blocks=1 << 40), BAD), (dict(nkv=0), BAD), (dict(cols=0), BAD), (dict(stride=3), BAD), (dict(B=-1), BAD),
    (dict(table=0), BAD), (dict(ctx=0), BAD), (dict(width=-1), BAD), (dict(rstride=3), BAD), (dict(first=-1), BAD), (dict(rows=0), BAD),
    (dict(counts=0), BAD), (dict(counts=FAKE + 2), ALIGN), (dict(lens=FAKE + 8), BAD), (dict(lens=FAKE + 256 + 40), BAD), (dict(lens=FAKE + 512), BAD),
    (dict(B=0), OK)])
def test_compact_status(L, over, want):
    assert status(L, "dspark_kv_compact", COMPACT, COMPACT_BASE, over) == want


FORK = "caches scales L blocks nkv bs D dt table stride cols pages lens R src dst n refs work bytes flags stream"
FORK_BASE = dict(caches=layers(FAKE), scales=None, L=1, blocks=4, nkv=2, bs=16, D=128, dt=0, table=FAKE, stride=4, cols=4, pages=FAKE + 256,
                 lens=FAKE + 512, R=3, src=FAKE + 768, dst=FAKE + 1024, n=2, refs=FAKE + 1280, work=FAKE + 4096, bytes=1 << 20, flags=0, stream=0)


@pytest.mark.parametrize("over,want", [
    (dict(L=-1), BAD), (dict(bs=0), BLOCK), (dict(blocks=0), BAD), (dict(cols=0), BAD), (dict(pages=0), BAD), (dict(lens=0), BAD), (dict(src=0), BAD),
    (dict(dst=0), BAD), (dict(refs=0), BAD), (dict(refs=FAKE + 1282), ALIGN), (dict(n=4097), BAD), (dict(n=-1), BAD), (dict(bytes=39), BAD),
    (dict(work=0), BAD), (dict(work=FAKE + 8), ALIGN), (dict(lens=FAKE + 256), BAD), (dict(dst=FAKE + 256), BAD), (dict(refs=FAKE + 16), BAD),
    (dict(n=0), OK), (dict(R=0), OK)])
def test_fork_status(L, over, want):
    assert status(L, "dspark_kv_fork", FORK, FORK_BASE, over) == want


RESIZE = "table stride cols pages tokens R refs blocks bs work bytes flags stream"
RESIZE_BASE = dict(table=FAKE, stride=4, cols=4, pages=FAKE + 256, tokens=FAKE + 512, R=3, refs=FAKE + 1024, blocks=9, bs=16, work=FAKE + 4096,
                   bytes=1 << 20, flags=0, stream=0)


@pytest.mark.parametrize("over,want", [
    (dict(bs=0), BLOCK), (dict(blocks=0), BAD), (dict(blocks=1 << 31), BAD), (dict(cols=0), BAD), (dict(stride=3), BAD), (dict(pages=0), BAD),
    (dict(tokens=0), BAD), (dict(refs=0), BAD), (dict(R=-1), BAD), (dict(bytes=51), BAD), (dict(work=0), BAD), (dict(work=FAKE + 8), ALIGN),
    (dict(tokens=FAKE + 256), BAD), (dict(refs=FAKE + 500), BAD), (dict(pages=FAKE + 32), BAD), (dict(R=0), OK)])
def test_resize_status(L, over, want):
    assert status(L, "dspark_kv_resize", RESIZE, RESIZE_BASE, over) == want


INSERT = "k kts khs v vts vhs T cache scales blocks nkv bs D table stride cols start ctx B flags stream"
INSERT_BASE = dict(k=FAKE, kts=256, khs=128, v=FAKE, vts=256, vhs=128, T=4, cache=FAKE, scales=FAKE, blocks=4, nkv=2, bs=16, D=128, table=FAKE,
                   stride=4, cols=4, start=FAKE, ctx=FAKE, B=2, flags=0, stream=0)


@pytest.mark.parametrize("over,want", [
    (dict(D=32), BAD), (dict(bs=0), BLOCK), (dict(cache=0), BAD), (dict(cache=FAKE + 8), ALIGN), (dict(kts=257), ALIGN), (dict(vhs=4), ALIGN),
    (dict(k=0), BAD), (dict(v=0), BAD), (dict(scales=0), BAD), (dict(start=0), BAD), (dict(ctx=0), BAD), (dict(k=FAKE + 8), ALIGN), (dict(T=-1), BAD),
    (dict(cols=0), BAD), (dict(T=0), OK), (dict(B=0), OK)])
def test_insert_status(L, over, want):
    assert status(L, "dspark_kv_insert_scaled", INSERT, INSERT_BASE, over) == want


ATTN = "q qts qhs T Hq Hkv D cache scales blocks bs table stride cols start ctx B kind mask words scale out lse work bytes flags stream"
ATTN_BASE = dict(q=FAKE, qts=512, qhs=128, T=4, Hq=4, Hkv=2, D=128, cache=FAKE, scales=FAKE, blocks=4, bs=16, table=FAKE, stride=4, cols=4,
                 start=FAKE, ctx=FAKE, B=2, kind=0, mask=0, words=0, scale=0.1, out=FAKE, lse=FAKE, work=FAKE, bytes=0, flags=0, stream=0)


@pytest.mark.parametrize("over,want", [
    (dict(D=32), BAD), (dict(Hq=3), BAD), (dict(scale=float("nan")), BAD), (dict(kind=3), BAD), (dict(kind=2), BAD), (dict(kind=2, words=1), BAD),
    (dict(scales=0), BAD), (dict(scales=FAKE + 1), ALIGN), (dict(out=0), BAD), (dict(lse=0), BAD), (dict(out=FAKE + 8), ALIGN),
    (dict(qts=511), ALIGN), (dict(cache=0), BAD), (dict(start=0), BAD), (dict(T=0), OK), (dict(B=0), OK)])
def test_scaled_attention_status(L, over, want):
    assert status(L, "dspark_tree_attention_scaled", ATTN, ATTN_BASE, over) == want


def test_workspace_queries(L):
    assert L.dspark_kv_fork_workspace(0) == 0 and L.dspark_kv_fork_workspace(-1) == -1 and L.dspark_kv_fork_workspace(4097) == -1
    assert L.dspark_kv_resize_workspace(0, 9) == 0 and L.dspark_kv_resize_workspace(5, 9) >= 60
    assert L.dspark_kv_resize_workspace(-1, 9) == -1 and L.dspark_kv_resize_workspace(5, 0) == -1 and L.dspark_kv_resize_workspace(5, 1 << 31) == -1
    assert L.dspark_tree_attention_scaled_workspace(0, 4, 2, 128, 3) == 0
    for bad in ((-1, 4, 2, 128, 3), (5, 3, 2, 128, 3), (5, 4, 2, 96, 3), (5, 4, 0, 128, 3), (5, 4, 2, 128, -3)):
        assert L.dspark_tree_attention_scaled_workspace(*bad) == -1


# ------------------------------------------------------------------ the Python layer


def refused(fn, *args, **kw):
    with pytest.raises(dk.DSparkError) as e:
        fn(*args, **kw)
    return str(e.value)


def ints(*n, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype)


def test_verify_refusals():
    base = dict(target_probs=torch.zeros((4, 10)), draft_tokens=ints(4, dtype=torch.int64), row_start=ints(2), uniforms=torch.zeros(4), max_accepted=3)
    for over, word in ((dict(target_probs=torch.zeros((4, 10)).half()), "fp32 or bf16"), (dict(target_probs=torch.zeros(4)), "rows, vocab"),
                       (dict(target_probs=torch.zeros((10, 4)).t()), "contiguous"), (dict(target_probs=None), "tensor"),
                       (dict(draft_probs=torch.zeros((4, 11))), "must be (4, 10)"), (dict(draft_probs=torch.zeros((3, 10))), "must be"),
                       (dict(draft_tokens=ints(4)), "int64"), (dict(draft_tokens=ints(3, dtype=torch.int64)), "4 rows"),
                       (dict(uniforms=torch.zeros(4).double()), "float32"), (dict(parents=ints(3)), "4 rows"), (dict(parents=ints(4, dtype=torch.int64)), "int32"),
                       (dict(row_start=ints(0)), "entry more"), (dict(max_accepted=0), "max_accepted"), (dict(max_accepted=1024), "max_accepted"),
                       (dict(tokens=ints(1, 3, dtype=torch.int64)), "(1, 4)"), (dict(rows=ints(1, 4)), "(1, 3)"), (dict(counts=ints(2)), "(1,)"),
                       (dict(error_flags=torch.zeros(1)), "error_flags"), ({}, "CUDA")):
        assert word in refused(dk.verify_drafts, **{**base, **over}), over


def test_page_refusals():
    cache, codes, scales = torch.zeros((4, 2, 16, 256)).bfloat16(), ints(4, 2, 16, 256, dtype=torch.uint8), ints(4, 2, 2, dtype=torch.int8)
    base = dict(kv_caches=[cache], block_table=ints(3, 2), context_lens=ints(3), rows=ints(3, 5), counts=ints(3))
    for over, word in ((dict(kv_caches=[]), "empty"), (dict(kv_caches=[None]), "tensors"), (dict(kv_caches=[cache, codes]), "kv_caches[1]"),
                       (dict(kv_caches=[cache, cache[:3]]), "kv_caches[1]"), (dict(block_scales=[scales]), "uint8"),
                       (dict(kv_caches=codes, block_scales=[scales, scales]), "2 block_scales"), (dict(kv_caches=codes, block_scales=scales[:3]), "shape"),
                       (dict(kv_caches=codes, block_scales=scales.int()), "int8"), (dict(rows=ints(2, 5)), "2 rows"), (dict(rows=ints(3)), "2 dims"),
                       (dict(counts=ints(2)), "counts"), (dict(new_lens=ints(4)), "new_lens"), (dict(first=-1), "first"), (dict(context_lens=ints(2)), "context_lens"),
                       ({}, "CUDA")):
        assert word in refused(dk.compact_kv, **{**base, **over}), over
    base = dict(kv_caches=cache, block_table=ints(3, 2), pages=ints(3), lens=ints(3), src=ints(1), dst=ints(1), refs=ints(4))
    for over, word in ((dict(pages=ints(2)), "requests"), (dict(lens=ints(2)), "lens"), (dict(dst=ints(2)), "dst"), (dict(refs=ints(5)), "refs"),
                       (dict(src=ints(4097), dst=ints(4097)), "4096"), (dict(src=ints(1, dtype=torch.int64)), "int32"), ({}, "CUDA")):
        assert word in refused(dk.fork_kv, **{**base, **over}), over
    base = dict(block_table=ints(3, 2), pages=ints(3), tokens=ints(3), refs=ints(4), block_size=16)
    for over, word in ((dict(refs=None), "refs"), (dict(tokens=ints(2)), "tokens"), (dict(block_size=0), "block_size"), (dict(block_size=1 << 31), "block_size"),
                       (dict(block_table=ints(3)), "block_table"), ({}, "CUDA")):
        assert word in refused(dk.resize_kv, **{**base, **over}), over


def test_scaled_refusals():
    cache, codes, scales = torch.zeros((4, 2, 16, 256)).bfloat16(), ints(4, 2, 16, 256, dtype=torch.uint8), ints(4, 2, 2, dtype=torch.int8)
    kv = torch.zeros((5, 2, 128)).bfloat16()
    base = dict(k=kv, v=kv, kv_cache=codes, block_scales=scales, block_table=ints(3, 2), query_start=ints(4), context_lens=ints(3))
    for over, word in ((dict(kv_cache=cache), "uint8"), (dict(k=kv.float()), "bfloat16"), (dict(v=kv[:4]), "v has shape"), (dict(k=kv[:, :1], v=kv[:, :1]), "heads"),
                       (dict(block_scales=scales[:, :1]), "contiguous"), (dict(block_scales=scales[:2]), "shape"), (dict(query_start=ints(3)), "query_start"), ({}, "CUDA")):
        assert word in refused(dk.insert_kv_scaled, **{**base, **over}), over
    q = torch.zeros((5, 4, 128)).bfloat16()
    for over, word in ((dict(kv_cache=cache), "uint8"), (dict(k_scale=torch.zeros(1)), "without k_scale"), (dict(block_scales=scales.float()), "int8"),
                       (dict(block_scales=scales[1:]), "shape"), ({}, "CUDA")):
        kw = {**dict(kv_cache=codes, block_scales=scales), **over}
        assert word in refused(dk.tree_attention, q, kw.pop("kv_cache"), ints(3, 2), ints(4), ints(3), **kw), over


# ------------------------------------------------------------------ the references themselves


def test_reference_codes():
    e = torch.tensor([[3, -5]], dtype=torch.int8)
    x = torch.tensor([[[1.0, 448 * 8.0, 3600.0, 0.3, -1.0, 14.0, 15.0, 2.0 ** -15]]], dtype=torch.float64)
    got = value(encode(x, e[:, None]), e[:, None])
    assert got[0, 0].tolist() == [1.0, 3584.0, 3584.0, 0.3125, -1.0, 14.0, 14.0, 2.0 ** -14 * 0]
    assert exponent(torch.tensor([[[448.0]], [[449.0]], [[0.0]], [[float("inf")]]], dtype=torch.float64)).tolist() == [0, 1, -32, -32]
    c = encode(x, e[:, None])
    assert torch.equal(grow(c, e, e), c)


def test_reference_walk_by_hand():
    """One drafted token over two: p = (3/4, 1/4), q = (1/4, 3/4)."""
    p, q = torch.tensor([[0.75, 0.25]] * 2), torch.tensor([[0.25, 0.75]] * 2)
    go = lambda tok, u0, u1: verify(p, q, torch.tensor([0, tok]), torch.tensor([0, 2]), None, torch.tensor([u0, u1]), 1, True)  # noqa: E731
    assert go(0, 0.8, 0.99)[0].tolist() == [[0, 1]]   # p >= q: accepted; the last from row 1's p
    assert go(1, 0.9, 0.32)[0].tolist() == [[1, 1]]   # accepted below 1/3
    assert go(1, 0.9, 0.34)[0].tolist() == [[0, -1]]  # the rest has token 0 alone
    pool = Pool(2, 3, 4, 4)
    pool.resize([5, 4])
    assert pool.table == [[0, 1, -1], [2, -1, -1]]
