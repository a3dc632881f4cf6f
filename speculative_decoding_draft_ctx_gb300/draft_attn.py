"""The operators on the caches that the context-KV writer fills: the cos|sin
table, rotary positions with the K/V insert, the drafted tokens' attention,
the attention weight each cached token received, and the eviction by it.

A draft step runs them in that order: ``rope_table`` once per model,
``rope_kv_insert`` (or ``qknorm_rope_kv_insert``) for the drafted tokens,
``tree_attention`` over the context and the drafted block,
``accumulate_attention_weight`` and, when a cache is over its budget,
``evict_kv``.  (DSpark draft model page: the draft layers rotate and insert
the draft tokens' K/V, then attend over ``[context | noise-block]``.)

Requests address their cached tokens through a block table: token j of
request b sits in block ``block_table[b, j // block_size]`` at offset
``j % block_size``.  Lengths, offsets and block numbers stay on the device;
what is out of range there is left out and raises a bit in ``error_flags``
(an int32 CUDA tensor of one element, if given).

``stream`` (a stream of the tensors' device, or its handle) runs the call
there; outputs that the call makes then belong to that stream.  The inputs are
used there without a record of it in PyTorch's allocator: the caller orders
that stream behind their producers and keeps them until the call has run (or
calls ``record_stream``).  Without it the current stream of the tensors'
device is used.
"""

from __future__ import annotations

import contextlib
import math

from ._binding import KV_BF16, KV_FP8_E4M3, DSparkError, check, lib

MASK_DENSE, MASK_CAUSAL, MASK_TREE = 0, 1, 2

torch = None  # loaded by the first call: an import statement per helper cost a call of a few tokens 4 us


def _load():
    global torch
    if torch is None:
        import torch


def _fail(message: str):
    raise DSparkError(1, message)


def _on(device, stream):
    """A context in which ``device`` and ``stream`` are current."""
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(device))
    if stream is not None:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        stack.enter_context(torch.cuda.stream(stream))
    return stack


def _elsewhere(device, stream) -> bool:
    """Whether a call has to change the current device or stream first."""
    if device.type != "cuda":
        _fail(f"tensors are on {device}, expected a CUDA device")
    if stream is not None and not isinstance(stream, int) and stream.device != device:
        _fail(f"stream is on {stream.device}, the tensors are on {device}")
    return stream is not None or device.index != torch.cuda.current_device()


def _current(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _tensor(name, x, dtype, device, ndim):
    """A contiguous tensor of this type, device and number of dims; its shape."""
    if not isinstance(x, torch.Tensor):
        _fail(f"{name} must be a tensor, got {type(x).__name__}")
    if x.dtype is not dtype:
        _fail(f"{name} must be {dtype}, got {x.dtype}")
    if x.device != device:
        _fail(f"{name} is on {x.device}, expected {device}")
    if not x.is_contiguous():
        _fail(f"{name} must be contiguous")
    if x.dim() != ndim:
        _fail(f"{name} must have {ndim} dims, got shape {tuple(x.shape)}")
    return x.shape


def _heads(name, x, device=None):
    """A bf16 [tokens, heads, head_dim] view with contiguous head rows; its shape."""
    if not isinstance(x, torch.Tensor):
        _fail(f"{name} must be a tensor, got {type(x).__name__}")
    if x.dtype is not torch.bfloat16:
        _fail(f"{name} must be {torch.bfloat16}, got {x.dtype}")
    if x.dim() != 3:
        _fail(f"{name} must have 3 dims (tokens, heads, head_dim), got shape {tuple(x.shape)}")
    if device is not None and x.device != device:
        _fail(f"{name} is on {x.device}, expected {device}")
    if x.shape[2] > 1 and x.stride(2) != 1:
        _fail(f"{name}'s head rows must be contiguous")
    return x.shape


def _scalar(name, x, device):
    if x is None:
        return 0
    if not isinstance(x, torch.Tensor) or x.dtype is not torch.float32 or x.device != device or x.numel() < 1:
        _fail(f"{name} must be an fp32 tensor of one element on {device}")
    return x.data_ptr()


def _flags(error_flags, device):
    if error_flags is None:
        return 0
    if (not isinstance(error_flags, torch.Tensor) or error_flags.dtype is not torch.int32 or error_flags.device != device
            or error_flags.numel() < 1):
        _fail(f"error_flags must be an int32 tensor of one element on {device}")
    return error_flags.data_ptr()


def _cache(kv_cache, device):
    """(num_blocks, num_kv_heads, block_size, head_dim, kv dtype) of a layer's cache."""
    if not isinstance(kv_cache, torch.Tensor) or kv_cache.dtype not in (torch.bfloat16, torch.uint8):
        _fail("kv_cache must be a bf16 or uint8 (fp8 e4m3) tensor")
    n, h, bs, row = _tensor("kv_cache", kv_cache, kv_cache.dtype, device, 4)
    if row not in (128, 256, 512):
        _fail(f"kv_cache rows hold {row} values: 2 * head_dim with head_dim 64, 128 or 256 expected")
    return n, h, bs, row // 2, KV_FP8_E4M3 if kv_cache.dtype is torch.uint8 else KV_BF16


def _block_scales(name, x, kv_cache):
    """The exponents of a page-scaled cache: int8, a pair per page and head."""
    shape = (kv_cache.shape[0], kv_cache.shape[1], 2)
    if _tensor(name, x, torch.int8, kv_cache.device, 3) != shape:
        _fail(f"{name} must have shape {shape}, got {tuple(x.shape)}")


def _table(block_table, context_lens, device):
    """(requests, table row stride, entries a row); the rows may be a column slice of a wider table."""
    if not isinstance(block_table, torch.Tensor) or block_table.dtype is not torch.int32 or block_table.dim() != 2:
        _fail("block_table must be an int32 tensor [requests, blocks]")
    if block_table.device != device:
        _fail(f"block_table is on {block_table.device}, expected {device}")
    B, n = block_table.shape
    stride = block_table.stride(0) if B > 1 else n
    if n < 1 or (n > 1 and block_table.stride(1) != 1) or stride < n:
        _fail("block_table must hold at least one entry a row, its rows contiguous and not overlapping")
    if _tensor("context_lens", context_lens, torch.int32, device, 1)[0] != B:
        _fail(f"context_lens has {context_lens.numel()} entries, {B} requests")
    return B, stride, n


# ------------------------------------------------------------------ rotary positions


def _frequencies(rotary_dim, theta, scaling):
    """``rope_frequencies`` with the frequencies as an fp64 array."""
    import numpy as np

    r, theta = int(rotary_dim), float(theta)
    if r < 2 or r % 2 or r > 512:
        raise DSparkError(2, f"rotary_dim {rotary_dim} must be even and in [2, 512]")
    if not (theta > 1.0 and math.isfinite(theta)):
        _fail(f"theta {theta} must be finite and above 1")
    i = np.arange(r // 2)
    f = theta ** (i * (-2.0 / r))
    if scaling is None:
        return f, 1.0
    s = dict(scaling)
    kind = s.pop("kind", None)
    factor = float(s.pop("factor", 0.0))
    if not (factor >= 1.0 and math.isfinite(factor)):
        _fail(f"scaling factor {factor} must be finite and at least 1")
    amplitude = 1.0
    if kind == "linear":
        f = f / factor
    elif kind in ("by_parts", "bands"):
        L = float(s.pop("original_positions", 0.0))
        if not (L >= 1.0 and math.isfinite(L)):
            _fail("scaling needs original_positions >= 1")
        if kind == "by_parts":
            fast, slow = float(s.pop("beta_fast", 32.0)), float(s.pop("beta_slow", 1.0))
            if not (fast > slow > 0.0 and math.isfinite(fast)):
                _fail("by_parts scaling needs beta_fast > beta_slow > 0, both finite")
            amplitude = float(s.pop("amplitude", 0.1 * math.log(factor) + 1.0))
            lo, hi = (r * math.log(L / (t * 2.0 * math.pi)) / (2.0 * math.log(theta)) for t in (fast, slow))
            lo, hi = max(0, math.floor(lo)), min(r - 1, math.ceil(hi))
            share = 1.0 - np.minimum(np.maximum((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            share[i >= hi] = 0.0  # hi <= 0: no dim turns more than beta_slow times
        else:
            low, high = float(s.pop("low_freq_factor", 1.0)), float(s.pop("high_freq_factor", 4.0))
            if not high > low:
                _fail("bands scaling needs high_freq_factor > low_freq_factor")
            share = np.minimum(np.maximum((f * (L / (2.0 * math.pi)) - low) / (high - low), 0.0), 1.0)
        f = f * (share + (1.0 - share) / factor)
    else:
        _fail(f"scaling kind {kind!r} unknown: linear, by_parts or bands")
    if s:
        _fail(f"scaling entries unknown to {kind}: {sorted(s)}")
    return f, amplitude


def rope_frequencies(rotary_dim, theta=10000.0, scaling=None):
    """(``rotary_dim / 2`` frequencies in radians per position, amplitude) of a
    cos|sin table.

    ``scaling`` is None or a dict with ``kind`` and ``factor`` (the context is
    ``factor`` times longer):

    * ``"linear"``: every frequency is divided by the factor.
    * ``"by_parts"``: with ``original_positions`` L, dims that turn at least
      ``beta_fast`` (32) times in L keep their frequency, those that turn at
      most ``beta_slow`` (1) times are divided by the factor, a linear ramp
      over the dim index lies between (its ends rounded outward); the table is
      multiplied by ``amplitude`` (0.1 ln factor + 1 if not given).
    * ``"bands"``: with ``original_positions`` L, a frequency that turns t
      times in L keeps the share (t - low) / (high - low), clamped to [0, 1],
      of itself and has the rest divided by the factor
      (``low_freq_factor`` 1, ``high_freq_factor`` 4).
    """
    f, amplitude = _frequencies(rotary_dim, theta, scaling)
    return f.tolist(), amplitude


def rope_table(num_positions, rotary_dim, theta=10000.0, scaling=None, first_position=0, dtype=None, device=None,
               out=None, stream=None):
    """The cos|sin table ``[num_positions, rotary_dim]`` (cos in the first
    half of a row) that the context-KV write, the inserts and
    ``rope_kv_insert`` read, for positions ``first_position`` onwards, made on
    the device: bf16 (the default; what the write and ``qknorm_rope_kv_insert``
    take) or fp32 (``rope_kv_insert`` takes both).  ``scaling``: see
    ``rope_frequencies``.  Angles are reduced exactly, so a far position loses
    only the frequency's own rounding (fp64) times the position."""
    _load()
    freqs, amplitude = _frequencies(rotary_dim, theta, scaling)
    n, r, first = int(num_positions), int(rotary_dim), int(first_position)
    if not (0 <= first <= 1 << 31 and 0 <= n <= (1 << 31) - first):  # ctypes cuts longer numbers off without a word
        _fail(f"num_positions {n} from {first}: positions in [0, 2^31) expected")
    if out is not None:
        if not isinstance(out, torch.Tensor) or out.dtype not in (torch.bfloat16, torch.float32):
            _fail("out must be a bf16 or fp32 tensor")
        if tuple(_tensor("out", out, out.dtype, out.device, 2)) != (n, r):
            _fail(f"out must have shape {(n, r)}, got {tuple(out.shape)}")
        if dtype is not None and dtype is not out.dtype:
            _fail(f"out is {out.dtype}, dtype {dtype}")
        device, dtype = out.device, out.dtype
    else:
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in (torch.bfloat16, torch.float32):
            _fail(f"dtype must be bf16 or fp32, got {dtype}")
        device = torch.device("cuda" if device is None else device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
    if _elsewhere(device, stream):
        with _on(device, stream):
            return rope_table(n, r, theta, scaling, first, dtype, device, out)
    if out is None:
        out = torch.empty((n, r), dtype=dtype, device=device)
    check(lib().dspark_rope_table(out.data_ptr(), first, n, r, freqs.__array_interface__["data"][0], amplitude,
                                  int(dtype is torch.float32), _current(device)))
    return out


def rope_kv_insert(q, k, cos_sin_cache, positions, rotary_dim, v=None, layout="half", inverse=False, slot_mapping=None,
                   kv_cache=None, k_scale=None, v_scale=None, q_out=None, k_out=None, error_flags=None, stream=None):
    """Rotary positions of ``q`` ``[T, num_heads, D]`` and ``k`` ``[T,
    num_kv_heads, D]`` (bf16 views with contiguous head rows, e.g. of a packed
    qkv), for drafts whose queries and keys take no norm; returns ``(q_out,
    k_out)``.  ``q_out=q``, ``k_out=k`` work in place.

    The leading ``rotary_dim`` dims turn at the token's position (table row
    ``cos_sin_cache[position]``, bf16 or fp32): ``layout="half"`` pairs dim i
    with i + rotary_dim / 2, ``"interleaved"`` dim 2i with 2i + 1.
    ``inverse=True`` turns back, which is also the rotation's gradient: the
    gradient of a loss with respect to ``q`` is this call on the gradient with
    respect to ``q_out``.

    With ``slot_mapping``, ``kv_cache`` and ``v``, tokens with a slot >= 0 have
    K' and V stored in the cache as the context-KV write stores them.  A token
    whose position is outside the table comes out unrotated, is not inserted
    and raises FLAG_POS_RANGE.
    """
    _load()
    T, Hq, D = _heads("q", q)
    dev = q.device
    Tk, Hkv, Dk = _heads("k", k, dev)
    if Tk != T or Dk != D:
        _fail(f"k has shape {tuple(k.shape)}, q {tuple(q.shape)}")
    if layout not in ("half", "interleaved"):
        _fail(f"layout {layout!r} unknown: half or interleaved")
    if not isinstance(cos_sin_cache, torch.Tensor) or cos_sin_cache.dtype not in (torch.bfloat16, torch.float32):
        _fail("cos_sin_cache must be a bf16 or fp32 tensor")
    rows, width = _tensor("cos_sin_cache", cos_sin_cache, cos_sin_cache.dtype, dev, 2)
    if width != rotary_dim or rows < 1:
        _fail(f"cos_sin_cache has shape {(rows, width)}, rotary_dim is {rotary_dim}")
    if _tensor("positions", positions, torch.int64, dev, 1)[0] < T:
        _fail(f"positions has {positions.numel()} entries, {T} tokens")
    num_blocks = block_size = 0
    kv_dtype = KV_BF16
    if (slot_mapping is None) != (kv_cache is None) or (slot_mapping is not None and v is None):
        _fail("slot_mapping, kv_cache and v go together")
    if slot_mapping is not None:
        num_blocks, nkv, block_size, hd, kv_dtype = _cache(kv_cache, dev)
        if nkv != Hkv or hd != D:
            _fail(f"kv_cache shape {tuple(kv_cache.shape)} does not match {Hkv} heads of {D}")
        if tuple(_heads("v", v, dev)) != (T, Hkv, D):
            _fail(f"v has shape {tuple(v.shape)}, k {tuple(k.shape)}")
        if _tensor("slot_mapping", slot_mapping, torch.int64, dev, 1)[0] < T:
            _fail(f"slot_mapping has {slot_mapping.numel()} entries, {T} tokens")
    for name, o, shape in (("q_out", q_out, (T, Hq, D)), ("k_out", k_out, (T, Hkv, D))):
        if o is not None and tuple(_heads(name, o, dev)) != shape:
            _fail(f"{name} has shape {tuple(o.shape)}, {shape} expected")
    flags = _flags(error_flags, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return rope_kv_insert(q, k, cos_sin_cache, positions, rotary_dim, v, layout, inverse, slot_mapping, kv_cache,
                                  k_scale, v_scale, q_out, k_out, error_flags)
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    if k_out is None:
        k_out = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=dev)
    insert = slot_mapping is not None
    vs = v.stride() if insert else (0, 0)
    qs, ks, qos, kos = q.stride(), k.stride(), q_out.stride(), k_out.stride()
    check(lib().dspark_rope_kv_insert(
        q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr() if insert else 0, vs[0], vs[1],
        q_out.data_ptr(), qos[0], qos[1], k_out.data_ptr(), kos[0], kos[1], cos_sin_cache.data_ptr(),
        int(cos_sin_cache.dtype is torch.float32), rows, positions.data_ptr(), T, Hq, Hkv, D, rotary_dim,
        int(layout == "interleaved"), int(bool(inverse)), slot_mapping.data_ptr() if insert else 0,
        kv_cache.data_ptr() if insert else 0, num_blocks, block_size, kv_dtype, _scalar("k_scale", k_scale, dev),
        _scalar("v_scale", v_scale, dev), flags, _current(dev)))
    return q_out, k_out


# ------------------------------------------------------------------ attention


def _queries(q, kv_cache, block_table, query_start, context_lens, scale):
    """What the attention and the weight accumulation check alike."""
    T, Hq, D = _heads("q", q)
    dev = q.device
    num_blocks, Hkv, block_size, hd, kv_dtype = _cache(kv_cache, dev)
    if hd != D or Hkv < 1 or Hq < 1 or Hq % Hkv:
        _fail(f"{Hq} query heads of {D} do not match kv_cache shape {tuple(kv_cache.shape)}")
    B, stride, entries = _table(block_table, context_lens, dev)
    if _tensor("query_start", query_start, torch.int32, dev, 1)[0] != B + 1:
        _fail(f"query_start has {query_start.numel()} entries, {B} requests")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    ts, hs, _ = q.stride()
    return (T, Hq, Hkv, D, B, dev, kv_dtype, scale,
            (q.data_ptr(), ts if T > 1 else 8, hs if Hq > 1 else 8, T, Hq, Hkv, D, kv_cache.data_ptr(), num_blocks,
             block_size, kv_dtype),
            (block_table.data_ptr(), stride, entries, query_start.data_ptr(), context_lens.data_ptr(), B))


def tree_attention(q, kv_cache, block_table, query_start, context_lens, tree_mask=None, causal=False, scale=None,
                   k_scale=None, v_scale=None, out=None, lse=None, error_flags=None, stream=None, block_scales=None):
    """The drafted tokens' attention over the paged cache; returns ``(out,
    lse)``: bf16 ``[T, num_heads, D]`` and fp32 ``[T, num_heads]`` (natural
    log; -inf, and zeros in ``out``, where a row sees nothing).  Scores and sums
    are fp32; the softmax weights enter the product with V as bf16 (as fp16 over
    an fp8 cache), so ``out`` is off by two bf16 roundings rather than one.

    ``q``: bf16 ``[T, num_heads, D]``, any token and head strides that are
    multiples of 8 elements; rows ``[query_start[b], query_start[b + 1])``
    (int32 ``[B + 1]``) are request b's drafted tokens.  ``kv_cache``: one
    layer's ``[num_blocks, num_kv_heads, block_size, 2 D]`` (bf16, or uint8
    e4m3 with the fp32 CUDA scalars ``k_scale`` / ``v_scale``); ``num_heads``
    is a multiple of ``num_kv_heads``.  ``block_table``: int32 ``[B, blocks]``.
    ``context_lens``: int32 ``[B]``; the drafted tokens' K/V have been inserted
    at the places behind the context.

    Every row sees the whole context.  Of its request's drafted tokens it sees
    all (the default: the drafter's dense block), itself and the earlier ones
    (``causal=True``), or token j where bit ``j % 64`` of ``tree_mask[t, j //
    64]`` is set (int64 ``[T, words]``).  Tokens that a row does not see do not
    reach its result, whatever they hold.  Rows that belong to no request are
    left as they were (uninitialised where this call makes the outputs).
    ``scale``: 1 / sqrt(D) if not given.

    ``block_scales``: int8 ``[num_blocks, num_kv_heads, 2]``, in the place of
    ``k_scale`` and ``v_scale``, for a page-scaled cache (uint8, as
    ``insert_kv_scaled`` fills it): the K and V of a page and head are its codes
    times 2 to these powers.
    """
    _load()
    T, Hq, Hkv, D, B, dev, kv_dtype, scale, head, table = _queries(q, kv_cache, block_table, query_start, context_lens,
                                                                  scale)
    kind, words = (MASK_CAUSAL, 0) if causal else (MASK_DENSE, 0)
    if tree_mask is not None:
        if causal:
            _fail("tree_mask and causal exclude each other")
        rows, words = _tensor("tree_mask", tree_mask, torch.int64, dev, 2)
        kind = MASK_TREE
        if rows != T or words < 1:
            _fail(f"tree_mask has shape {(rows, words)}, {T} rows of at least one word expected")
    if out is not None and tuple(_tensor("out", out, torch.bfloat16, dev, 3)) != (T, Hq, D):
        _fail(f"out must have shape {(T, Hq, D)}, got {tuple(out.shape)}")
    if lse is not None and tuple(_tensor("lse", lse, torch.float32, dev, 2)) != (T, Hq):
        _fail(f"lse must have shape {(T, Hq)}, got {tuple(lse.shape)}")
    ks, vs, flags = _scalar("k_scale", k_scale, dev), _scalar("v_scale", v_scale, dev), _flags(error_flags, dev)
    if block_scales is not None:
        if kv_dtype != KV_FP8_E4M3 or k_scale is not None or v_scale is not None:
            _fail("block_scales go with a uint8 cache, without k_scale and v_scale")
        _block_scales("block_scales", block_scales, kv_cache)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return tree_attention(q, kv_cache, block_table, query_start, context_lens, tree_mask, causal, scale, k_scale,
                                  v_scale, out, lse, error_flags, None, block_scales)
    if out is None:
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    L = lib()
    # the partial results of requests that are split over CTAs: made anew by
    # each call, on its stream (or in the graph's own pool), so calls never share it
    # (a size below 0: the call refuses the same sizes, with its status)
    size = max(0, L.dspark_tree_attention_workspace(T, Hq, Hkv, D, B, kv_dtype) if block_scales is None else
               L.dspark_tree_attention_scaled_workspace(T, Hq, Hkv, D, B))
    work = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    rest = (*table, kind, tree_mask.data_ptr() if words else 0, words, scale, out.data_ptr(), lse.data_ptr(),
            work.data_ptr() if size else 0, size, flags, _current(dev))
    if block_scales is None:
        check(L.dspark_tree_attention(*head, ks, vs, *rest))
    else:
        check(L.dspark_tree_attention_scaled(*head[:8], block_scales.data_ptr(), *head[8:10], *rest))
    return out, lse


def accumulate_attention_weight(q, kv_cache, block_table, query_start, context_lens, lse, weights, decay=1.0, scale=None,
                                k_scale=None, error_flags=None, stream=None):
    """Adds to ``weights`` (fp32 ``[B, num_kv_heads, places]``, in place, also
    returned) the attention weight that every context token received from the
    drafted tokens' queries, summed over a KV head's query heads, after
    multiplying the old value by ``decay``; places behind a request's context
    stay.  ``lse`` is what ``tree_attention`` returned for the same arguments
    (the other arguments are as there)."""
    _load()
    T, Hq, Hkv, D, B, dev, kv_dtype, scale, head, table = _queries(q, kv_cache, block_table, query_start, context_lens,
                                                                  scale)
    if tuple(_tensor("lse", lse, torch.float32, dev, 2)) != (T, Hq):
        _fail(f"lse must have shape {(T, Hq)}, got {tuple(lse.shape)}")
    rows, heads, places = _tensor("weights", weights, torch.float32, dev, 3)
    if rows != B or heads != Hkv:
        _fail(f"weights must have shape {(B, Hkv, '*')}, got {tuple(weights.shape)}")
    ks, flags = _scalar("k_scale", k_scale, dev), _flags(error_flags, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return accumulate_attention_weight(q, kv_cache, block_table, query_start, context_lens, lse, weights, decay,
                                               scale, k_scale, error_flags)
    check(lib().dspark_attention_weight_accumulate(*head, ks, *table, lse.data_ptr(), scale, float(decay),
                                                   weights.data_ptr(), places, flags, _current(dev)))
    return weights


# ------------------------------------------------------------------ eviction


def evict_kv(kv_cache, block_table, context_lens, weights, token_positions, seq_lens, budget, sinks=0, recent=0,
             weights_out=None, positions_out=None, new_lens=None, error_flags=None, stream=None):
    """Cuts every request's context down to its ``budget`` heaviest tokens per
    KV head, in one layer's cache; returns the new lengths (int32 ``[B]``,
    ``min(context_lens, budget)``).

    ``weights`` (fp32) and ``token_positions`` (int32, the sequence position of
    the token at each place) are ``[B, num_kv_heads, places]``.  Tokens at
    positions below ``sinks`` and at or above ``seq_lens[b] - recent`` stay in
    any case (``sinks + recent <= budget``); of the others the heaviest stay,
    the one at the lower place where weights are equal, NaN last.  Kept tokens
    from places >= budget move into the places that were given up, the first
    into the first: the order of the others is kept, and only as many rows
    move as there are gaps.  ``weights_out`` and ``positions_out`` receive the
    weights and positions of the new places (the inputs themselves, in place,
    if not given; places behind the new length hold 0 and -1 up to the old
    one).  Each KV head keeps its own tokens, so requests must not share
    blocks.  Layers keep different tokens: call it once per layer, with that
    layer's weights and positions.  ``new_lens=context_lens`` updates the
    lengths in place (in the last layer's call: the others need the old ones).
    """
    _load()
    if not isinstance(kv_cache, torch.Tensor):
        _fail("kv_cache must be a bf16 or uint8 (fp8 e4m3) tensor")
    dev = kv_cache.device
    num_blocks, Hkv, block_size, D, kv_dtype = _cache(kv_cache, dev)
    B, stride, entries = _table(block_table, context_lens, dev)
    shape = tuple(_tensor("weights", weights, torch.float32, dev, 3))
    if shape[:2] != (B, Hkv):
        _fail(f"weights must have shape {(B, Hkv, '*')}, got {shape}")
    if tuple(_tensor("token_positions", token_positions, torch.int32, dev, 3)) != shape:
        _fail(f"token_positions must have shape {shape}, got {tuple(token_positions.shape)}")
    if _tensor("seq_lens", seq_lens, torch.int32, dev, 1)[0] != B:
        _fail(f"seq_lens has {seq_lens.numel()} entries, {B} requests")
    if weights_out is None:
        weights_out = weights
    elif tuple(_tensor("weights_out", weights_out, torch.float32, dev, 3)) != shape:
        _fail(f"weights_out must have shape {shape}, got {tuple(weights_out.shape)}")
    if positions_out is None:
        positions_out = token_positions
    elif tuple(_tensor("positions_out", positions_out, torch.int32, dev, 3)) != shape:
        _fail(f"positions_out must have shape {shape}, got {tuple(positions_out.shape)}")
    if new_lens is not None and _tensor("new_lens", new_lens, torch.int32, dev, 1)[0] != B:
        _fail(f"new_lens has {new_lens.numel()} entries, {B} requests")
    flags = _flags(error_flags, dev)
    budget, sinks, recent = int(budget), int(sinks), int(recent)
    if budget < 1 or sinks < 0 or recent < 0 or sinks + recent > budget:
        _fail(f"budget {budget}, sinks {sinks}, recent {recent}: 0 <= sinks + recent <= budget, budget >= 1 expected")
    # beyond any length and position; ctypes cuts numbers of more than 64 bits off without a word
    budget, sinks, recent = min(budget, 1 << 62), min(sinks, 1 << 60), min(recent, 1 << 60)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return evict_kv(kv_cache, block_table, context_lens, weights, token_positions, seq_lens, budget, sinks, recent,
                            weights_out, positions_out, new_lens, error_flags)
    if new_lens is None:
        new_lens = torch.empty(B, dtype=torch.int32, device=dev)
    L = lib()
    size = max(0, L.dspark_kv_evict_workspace(B, Hkv, shape[2], budget))
    work = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    check(L.dspark_kv_evict(kv_cache.data_ptr(), num_blocks, Hkv, block_size, D, kv_dtype, block_table.data_ptr(), stride,
                            entries, context_lens.data_ptr(), B, weights.data_ptr(), token_positions.data_ptr(),
                            weights_out.data_ptr(), positions_out.data_ptr(), shape[2], seq_lens.data_ptr(), budget, sinks,
                            recent, new_lens.data_ptr(), work.data_ptr() if size else 0, size, flags, _current(dev)))
    return new_lens
