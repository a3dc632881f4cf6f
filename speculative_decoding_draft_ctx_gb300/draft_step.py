"""What a serving loop does around the target's run over the drafted tokens:
``verify_drafts`` decides which of them stand, ``compact_kv`` moves the
accepted path's K/V behind the context, ``resize_kv`` gives pages back to the
pool and takes the next step's, ``fork_kv`` lets one request's cache continue
as several, and ``insert_kv_scaled`` fills a page-scaled cache (8-bit codes
with one power-of-two scale per page and head), which ``tree_attention`` reads
with ``block_scales``.  (``accumulate_attention_weight``, ``evict_kv`` and the
context-KV writes take caches with per-tensor scales only.)

No call needs a length on the host, so a whole step can be captured into a
CUDA graph.  Caches, block tables, ``error_flags`` and ``stream`` are as in
``tree_attention`` and the other operators on the caches: lengths, rows and
pages out of range are left out and raise a bit in ``error_flags``.  A page is
a block of the cache: ``block_size`` tokens of every head, in every layer.

The page pool is an int32 tensor ``refs`` ``[num_blocks]``: how many block table
entries hold the page; 0 is free.  Pages are given out lowest number first.
"""

from __future__ import annotations

from array import array

from . import draft_attn as _da
from ._binding import KV_FP8_E4M3, check, lib
from .draft_attn import _block_scales, _cache, _current, _elsewhere, _fail, _flags, _heads, _on, _table, _tensor


torch = None  # loaded by the first call, as in draft_attn


def _load():
    global torch
    if torch is None:
        _da._load()
        torch = _da.torch


# A call of a few tokens is bound by its host side, most of which are the checks of
# its arguments: `_is` answers for all that is right with one in a third of the
# time of those that name what is wrong (verify_drafts 25 -> 17 us).
def _is(x, dtype, device, shape):
    """Whether x is a contiguous tensor of exactly this type, device and shape."""
    return isinstance(x, torch.Tensor) and x.dtype is dtype and x.shape == shape and x.device == device and x.is_contiguous()


def _ints(name, x, n, device):
    if not _is(x, torch.int32, device, (n,)) and _tensor(name, x, torch.int32, device, 1)[0] != n:
        _fail(f"{name} has {x.numel()} entries, {n} expected")


def _whole(name, x, lo, hi):
    x = int(x)
    if not lo <= x <= hi:
        _fail(f"{name} {x} not in [{lo}, {hi}]")
    return x


# ------------------------------------------------------------------ verification


def _probabilities(name, x, device=None, shape=None):
    """fp32 or bf16 rows with contiguous entries: (dtype code, row stride)."""
    if not isinstance(x, torch.Tensor):
        _fail(f"{name} must be a tensor, got {type(x).__name__}")
    if x.dtype not in (torch.float32, torch.bfloat16):
        _fail(f"{name} must be fp32 or bf16, got {x.dtype}")
    if x.dim() != 2 or (shape is not None and x.shape != shape):
        _fail(f"{name} must be {tuple(shape) if shape else '[rows, vocab]'}, got shape {tuple(x.shape)}")
    if device is not None and x.device != device:
        _fail(f"{name} is on {x.device}, expected {device}")
    (rows, width), (row, each) = x.shape, x.stride()
    if each != 1 and width > 1:
        _fail(f"{name}'s rows must be contiguous")
    return int(x.dtype is torch.bfloat16), row if rows > 1 else width


def verify_drafts(target_probs, draft_tokens, row_start, uniforms, max_accepted, draft_probs=None, parents=None,
                  replacement=True, tokens=None, rows=None, counts=None, error_flags=None, stream=None):
    """Which drafted tokens the target accepts, and the token behind them, so
    that what comes out is distributed as the target's own; returns ``(tokens,
    rows, counts)``.

    Request b's rows are ``[row_start[b], row_start[b + 1])`` (int32 ``[B + 1]``):
    its row 0 is the last accepted token, each other one a drafted token
    (``draft_tokens``, int64 ``[T]``), drawn behind row ``parents[i] < i`` of its
    request (int32 ``[T]``; None: behind the row before, a chain).  Row r of
    ``target_probs`` and ``draft_probs`` (fp32 or bf16 ``[T, vocab]``, any row
    stride) is the distribution of the token behind row r; entries outside
    [0, 1] count as the nearer end, NaN as 0.  ``uniforms``: fp32 ``[T]``, in
    [0, 1).

    From row 0 on, the children of the row reached are tested in row order:
    child x stands where ``u_x q(x) Z < R(x)``, with R = p and Z = 1 at first;
    each rejection takes ``Z q`` from R (cut off at 0) and makes Z its sum.
    ``replacement=False``: a row's children are distinct, drawn one after
    another, and q leaves the rejected ones out.  ``draft_probs=None``: the drafter
    takes its tokens without drawing; a rejected one leaves R and Z.  Where no
    child stands, or after ``max_accepted`` tokens (1 to 1023), the last token is
    the first whose cumulated R exceeds ``u_0 sum R``.

    ``tokens``: int64 ``[B, max_accepted + 1]``, the accepted tokens, the last
    one, then -1; ``rows``: int32 ``[B, max_accepted]``, the accepted tokens' rows
    (what ``compact_kv`` takes), then -1; ``counts``: int32 ``[B]``, how many
    stand.  Made by the call if not given; refused where they overlap one another or
    an input.  A request has up to 1024 rows; one without rows gets -1 and 0.  FLAG_ROW: a token outside the vocabulary
    (rejected), a parent that is not a row before it (never tested), or a last row
    without any probability (token -1).
    """
    _load()
    pt, ps = _probabilities("target_probs", target_probs)
    T, V = shape = target_probs.shape
    dev = target_probs.device
    dt, ds = (0, 0) if draft_probs is None else _probabilities("draft_probs", draft_probs, dev, shape)
    if not (_is(draft_tokens, torch.int64, dev, (T,)) and _is(uniforms, torch.float32, dev, (T,)) and
            (parents is None or _is(parents, torch.int32, dev, (T,)))):
        for name, x, dtype in (("draft_tokens", draft_tokens, torch.int64), ("uniforms", uniforms, torch.float32),
                               *((("parents", parents, torch.int32),) if parents is not None else ())):
            if _tensor(name, x, dtype, dev, 1)[0] != T:
                _fail(f"{name} has {x.numel()} entries, {T} rows")
    B = _tensor("row_start", row_start, torch.int32, dev, 1)[0] - 1
    if B < 0:
        _fail("row_start must have an entry more than there are requests")
    n = _whole("max_accepted", max_accepted, 1, 1023)
    if tokens is not None or rows is not None or counts is not None:
        for name, x, dtype, shape in (("tokens", tokens, torch.int64, (B, n + 1)), ("rows", rows, torch.int32, (B, n)),
                                      ("counts", counts, torch.int32, (B,))):
            if x is not None and tuple(_tensor(name, x, dtype, dev, len(shape))) != shape:
                _fail(f"{name} must have shape {shape}, got {tuple(x.shape)}")
    flags = _flags(error_flags, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return verify_drafts(target_probs, draft_tokens, row_start, uniforms, n, draft_probs, parents, replacement,
                                 tokens, rows, counts, error_flags)
    if tokens is None:
        tokens = torch.empty((B, n + 1), dtype=torch.int64, device=dev)
    if rows is None:
        rows = torch.empty((B, n), dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty(B, dtype=torch.int32, device=dev)
    check(lib().dspark_verify_drafts(
        target_probs.data_ptr(), pt, ps, 0 if draft_probs is None else draft_probs.data_ptr(), dt, ds, T, V,
        draft_tokens.data_ptr(), 0 if parents is None else parents.data_ptr(), uniforms.data_ptr(), row_start.data_ptr(), B,
        n, int(bool(replacement)), tokens.data_ptr(), rows.data_ptr(), counts.data_ptr(), flags, _current(dev)))
    return tokens, rows, counts


# ------------------------------------------------------------------ pages


def _layers(kv_caches, block_scales):
    """(device, host arrays, the caches as the calls take them): layers alike."""
    caches = [kv_caches] if isinstance(kv_caches, torch.Tensor) else list(kv_caches)
    if not caches:
        _fail("kv_caches is empty")
    if not isinstance(caches[0], torch.Tensor):
        _fail(f"kv_caches must be tensors, got {type(caches[0]).__name__}")
    dev, shape, dtype = caches[0].device, caches[0].shape, caches[0].dtype
    blocks, H, bs, D, kv_dtype = _cache(caches[0], dev)
    for i in range(1, len(caches)):
        if not _is(caches[i], dtype, dev, shape):
            _fail(f"kv_caches[{i}] is not like kv_caches[0]: {dtype} of shape {tuple(shape)} on {dev}, contiguous")
    L = len(caches)
    scales = None
    if block_scales is not None:
        if kv_dtype != KV_FP8_E4M3:
            _fail("block_scales go with uint8 caches")
        scales = [block_scales] if isinstance(block_scales, torch.Tensor) else list(block_scales)
        if len(scales) != L:
            _fail(f"{len(scales)} block_scales, {L} caches")
        pairs = (blocks, H, 2)
        for i, x in enumerate(scales):
            if not _is(x, torch.int8, dev, pairs):
                _block_scales(f"block_scales[{i}]", x, caches[0])
    # host arrays of addresses; the call keeps them (`hold`) until it has read them
    hold = array("Q", [x.data_ptr() for x in caches])
    at, scales_at = hold.buffer_info()[0], 0
    if scales is not None:
        hold = (hold, array("Q", [x.data_ptr() for x in scales]))
        scales_at = hold[1].buffer_info()[0]
    return dev, hold, (at, scales_at, L, blocks, H, bs, D, kv_dtype)


def compact_kv(kv_caches, block_table, context_lens, rows, counts, first=1, block_scales=None, new_lens=None,
               error_flags=None, stream=None):
    """Moves the accepted tokens' K/V together, in every layer of ``kv_caches`` (a
    tensor or a list of them): of request b, the token at place
    ``context_lens[b] + rows[b, j]`` goes to ``context_lens[b] + first + j`` for
    j < ``counts[b]``; returns the new lengths, ``context_lens + first +
    counts`` (int32 ``[B]``; ``new_lens`` if given, which must not overlap the
    inputs).

    ``rows`` (int32 ``[B, width]``) and ``counts`` (int32 ``[B]``) are what
    ``verify_drafts`` returned: rows ascend and lie at or behind ``first + j``.
    ``first=1``: row 0 is the last accepted token, whose K/V stays.  (A request that
    had no rows in the step grows by ``first`` too: keep its old length.)  Requests must
    not share the pages that rows move into.  ``block_scales`` (int8 ``[num_blocks,
    num_kv_heads, 2]`` per layer): page-scaled caches; a page's scale grows to the
    largest that comes in, and what the page holds is encoded anew.
    """
    _load()
    dev, hold, layers = _layers(kv_caches, block_scales)
    B, stride, entries = _table(block_table, context_lens, dev)
    R, width = _tensor("rows", rows, torch.int32, dev, 2)
    if R != B:
        _fail(f"rows has {R} rows, {B} requests")
    _ints("counts", counts, B, dev)
    if new_lens is not None:
        _ints("new_lens", new_lens, B, dev)
    first = _whole("first", first, 0, 1 << 30)
    flags = _flags(error_flags, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return compact_kv(kv_caches, block_table, context_lens, rows, counts, first, block_scales, new_lens, error_flags)
    if new_lens is None:
        new_lens = torch.empty(B, dtype=torch.int32, device=dev)
    check(lib().dspark_kv_compact(*layers, block_table.data_ptr(), stride, entries, context_lens.data_ptr(), B, rows.data_ptr(),
                                  width, width, counts.data_ptr(), first, new_lens.data_ptr(), flags, _current(dev)))
    return new_lens


def fork_kv(kv_caches, block_table, pages, lens, src, dst, refs, block_scales=None, error_flags=None, stream=None):
    """Makes row ``dst[i]`` of the block table a copy of row ``src[i]``, for all i:
    the pages full of its tokens are shared (``refs`` + 1), a last page that is
    not full is copied into a free one, in every layer of ``kv_caches`` (a tensor
    or a list); pages that ``src`` holds beyond its tokens stay its own.

    In place: ``block_table`` (int32 ``[R, blocks]``), ``pages`` (int32 ``[R]``: the
    entries that a row holds), ``lens`` (int32 ``[R]``: its tokens), ``refs`` (int32
    ``[num_blocks]``).  ``src``, ``dst``: int32, up to 4096 pairs.  A row may be
    the ``src`` of several pairs.  Left out: a pair whose ``dst`` holds pages, is a
    ``src`` of the call or the ``dst`` of an earlier pair, or that has a row or
    length out of range (FLAG_LENGTH), and one for whose last page there is no
    free one (FLAG_PAGES; they are given out in the order of the pairs).
    """
    _load()
    dev, hold, layers = _layers(kv_caches, block_scales)
    R, stride, entries = _table(block_table, pages, dev)
    _ints("lens", lens, R, dev)
    n = _tensor("src", src, torch.int32, dev, 1)[0]
    _ints("dst", dst, n, dev)
    _ints("refs", refs, layers[3], dev)
    if n > 4096:
        _fail(f"{n} pairs, at most 4096 a call")
    flags = _flags(error_flags, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return fork_kv(kv_caches, block_table, pages, lens, src, dst, refs, block_scales, error_flags)
    L = lib()
    size = L.dspark_kv_fork_workspace(n)
    work = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    check(L.dspark_kv_fork(*layers, block_table.data_ptr(), stride, entries, pages.data_ptr(), lens.data_ptr(), R, src.data_ptr(),
                           dst.data_ptr(), n, refs.data_ptr(), work.data_ptr() if size else 0, size, flags, _current(dev)))


def resize_kv(block_table, pages, tokens, refs, block_size, error_flags=None, stream=None):
    """Gives every row r of the block table the pages of ``tokens[r]`` tokens
    (int32 ``[R]``): entries beyond them go back to the pool (and become -1), then
    missing ones are taken, in the order of the rows.  0 tokens frees a row.

    In place: ``block_table`` (int32 ``[R, blocks]``), ``pages`` (int32 ``[R]``: the
    entries that a row holds), ``refs`` (int32 ``[num_blocks]``).  A row is served
    where the pages that it and all rows before it ask for are there; the others
    keep what they hold (FLAG_PAGES).  A row whose tokens do not fit the table
    keeps its pages (FLAG_LENGTH).  FLAG_REFS: a page given back that nobody held.
    """
    _load()
    if not isinstance(refs, torch.Tensor):
        _fail(f"refs must be a tensor, got {type(refs).__name__}")
    dev = refs.device
    blocks = _tensor("refs", refs, torch.int32, dev, 1)[0]
    R, stride, entries = _table(block_table, pages, dev)
    _ints("tokens", tokens, R, dev)
    block_size = _whole("block_size", block_size, 1, (1 << 31) - 1)
    flags = _flags(error_flags, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return resize_kv(block_table, pages, tokens, refs, block_size, error_flags)
    L = lib()
    size = max(0, L.dspark_kv_resize_workspace(R, blocks))
    work = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    check(L.dspark_kv_resize(block_table.data_ptr(), stride, entries, pages.data_ptr(), tokens.data_ptr(), R, refs.data_ptr(), blocks,
                             block_size, work.data_ptr() if size else 0, size, flags, _current(dev)))


# ------------------------------------------------------------------ page-scaled caches


def insert_kv_scaled(k, v, kv_cache, block_scales, block_table, query_start, context_lens, error_flags=None, stream=None):
    """Stores the new tokens' ``k`` and ``v`` (bf16 ``[T, num_kv_heads, D]`` views,
    strides multiples of 8 elements) in a page-scaled cache (uint8 ``[num_blocks,
    num_kv_heads, block_size, 2 D]``, ``block_scales`` int8 ``[num_blocks,
    num_kv_heads, 2]``), in place: rows ``[query_start[b], query_start[b + 1])``
    go to the places behind request b's ``context_lens[b]`` tokens.

    A page's scale is the least power of two 2^e, e in [-32, 31], with |x| <= 448 *
    2^e for the finite new values of the page and head, K and V apart; a page
    that already holds context tokens keeps its scale or has it grow, its codes
    encoded anew.  Codes are e4m3 of x / 2^e, saturating, NaN kept.  Pages that
    tokens go into belong to one request.
    """
    _load()
    T, H, D = _heads("k", k)
    dev = k.device
    if _heads("v", v, dev) != (T, H, D):
        _fail(f"v has shape {tuple(v.shape)}, k {tuple(k.shape)}")
    blocks, nkv, bs, hd, kv_dtype = _cache(kv_cache, dev)
    if kv_dtype != KV_FP8_E4M3:
        _fail("a page-scaled cache is uint8")
    if nkv != H or hd != D:
        _fail(f"kv_cache shape {tuple(kv_cache.shape)} does not match {H} heads of {D}")
    _block_scales("block_scales", block_scales, kv_cache)
    B, stride, entries = _table(block_table, context_lens, dev)
    _ints("query_start", query_start, B + 1, dev)
    flags = _flags(error_flags, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return insert_kv_scaled(k, v, kv_cache, block_scales, block_table, query_start, context_lens, error_flags)
    ks, vs = k.stride(), v.stride()
    one = lambda s: (s[0] if T > 1 else 8, s[1] if H > 1 else 8)  # noqa: E731  (strides of single entries mean nothing)
    check(lib().dspark_kv_insert_scaled(k.data_ptr(), *one(ks), v.data_ptr(), *one(vs), T, kv_cache.data_ptr(),
                                        block_scales.data_ptr(), blocks, H, bs, D, block_table.data_ptr(), stride, entries,
                                        query_start.data_ptr(), context_lens.data_ptr(), B, flags, _current(dev)))
