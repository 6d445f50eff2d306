"""A paged cache of keys and values held in 8 bits, and softmax attention over it: binding of
gdr_page_*, gdr_cache_append and gdr_cache_attn (gdr.h).

    plan = page_plan(block_table, kv_lens, free_pages, free_count, page)   # the next token of every request
    q, k = rotary_fwd(q, k, plan.positions, rates)
    cache_append(k, v, plan.slots, k_cache, v_cache, k_scale, v_scale)
    o = cache_attn(q, k_cache, v_cache, k_scale, v_scale, block_table, plan.kv_lens)

k_cache and v_cache are [num_pages, kv_heads, page, d] in torch.float8_e4m3fn or torch.int8, k_scale
and v_scale [num_pages, kv_heads] fp32. Everything stays on the device: a step can be captured
into a graph. Argument marshalling only.
"""
import collections
import ctypes
import functools

import torch

from . import ops
from .described import dense, describe, named, new_like, rows_stride
from .linattn import _addr
from .ops import _DTYPES, _launch, _need

_CODES = {torch.float8_e4m3fn: 0, torch.int8: 1}

PagePlan = collections.namedtuple("PagePlan", "kv_lens free_count cu_q start positions slots")


class PageShape(ctypes.Structure):
    """struct gdr_page_shape of gdr.h."""
    _fields_ = [("num_seqs", ctypes.c_int64), ("width", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("num_pages", ctypes.c_int64), ("page", ctypes.c_int)]


class CacheShape(ctypes.Structure):
    """struct gdr_cache_shape of gdr.h."""
    _fields_ = [("num_pages", ctypes.c_int64), ("kv_heads", ctypes.c_int), ("page", ctypes.c_int),
                ("d", ctypes.c_int), ("codes", ctypes.c_int), ("dtype", ctypes.c_int)]


class CacheAttnShape(ctypes.Structure):
    """struct gdr_cache_attn_shape of gdr.h."""
    _fields_ = [("cache", CacheShape), ("num_seqs", ctypes.c_int64), ("total_tokens", ctypes.c_int64),
                ("max_q", ctypes.c_int64), ("width", ctypes.c_int64), ("q_stride", ctypes.c_int64),
                ("heads", ctypes.c_int), ("causal", ctypes.c_int), ("scale", ctypes.c_float),
                ("softcap", ctypes.c_float)]


def _opt(t, name):
    return None if t is None else describe(t, name)


def _table(t):
    dense(t, "block_table", torch.int32)
    if len(t.shape) != 2:
        raise ValueError("block_table must have shape [num_seqs, width]")
    return t.device, t.shape[0], t.shape[1]


@functools.lru_cache(maxsize=256)
def _checked_plan(block_table, kv_lens, free_pages, free_count, q_lens, rows, page, outs):
    block_table, kv_lens, free_pages, free_count, q_lens = named(block_table, kv_lens, free_pages, free_count, q_lens)
    outs = named(*outs)
    dev, n, width = _table(block_table)
    i32 = torch.int32
    dense(kv_lens, "kv_lens", i32, dev, (n,))
    dense(free_pages, "free_pages", i32, dev)
    dense(free_count, "free_count", i32, dev, (1,))
    if q_lens is not None:
        dense(q_lens, "q_lens", i32, dev, (n,))
        if rows is None:
            raise ValueError("q_lens needs rows, the tokens of the packed batch")
    rows = n if rows is None else rows
    if rows < 0:
        raise ValueError(f"rows must not be negative, got {rows}")
    sizes = (n, 1, n + 1, n, rows, rows)
    for t, name, size in zip(outs, ("kv_lens_out", "free_count_out", "cu_q", "start", "positions", "slots"), sizes):
        if t is not None:
            dense(t, name, i32, dev, (size,))
    return ctypes.byref(PageShape(n, width, rows, free_pages.shape.numel(), page)), sizes


def page_plan(block_table, kv_lens, free_pages, free_count, page, q_lens=None, rows=None, kv_lens_out=None,
              free_count_out=None, cu_q=None, start=None, positions=None, slots=None, stream=None):
    """Pages, positions and slots of the requests' new tokens (gdr_page_plan): block_table
    [num_seqs, width], kv_lens [num_seqs], free_pages [num_pages] and free_count [1] int32; q_lens
    [num_seqs] int32 or None for one token each; rows: tokens of the packed batch, padding included
    (default num_seqs; needed with q_lens). The table gets its new entries in place. Returns a
    PagePlan (kv_lens, free_count, cu_q, start, positions, slots) of new tensors or those
    given; kv_lens_out may be kv_lens and free_count_out may be free_count. start is -1 for a refused request."""
    lib = ops._load()
    outs = (kv_lens_out, free_count_out, cu_q, start, positions, slots)
    shape, sizes = _checked_plan(
        describe(block_table, "block_table"), describe(kv_lens, "kv_lens"), describe(free_pages, "free_pages"),
        describe(free_count, "free_count"), _opt(q_lens, "q_lens"), None if rows is None else int(rows), int(page),
        tuple([None if t is None else describe(t, "an output") for t in outs]))
    outs = [new_like(kv_lens, stream, (n,)) if t is None else t for t, n in zip(outs, sizes)]
    _launch(lib.gdr_page_plan, "gdr_page_plan", kv_lens.device, stream, shape, _addr(q_lens), kv_lens.data_ptr(),
            free_pages.data_ptr(), free_count.data_ptr(), block_table.data_ptr(), *[t.data_ptr() for t in outs])
    return PagePlan(*outs)


@functools.lru_cache(maxsize=256)
def _checked_release(block_table, kv_lens, done, free_pages, free_count, page):
    block_table, kv_lens, done, free_pages, free_count = named(block_table, kv_lens, done, free_pages, free_count)
    dev, n, width = _table(block_table)
    dense(kv_lens, "kv_lens", torch.int32, dev, (n,))
    if done.dtype not in (torch.bool, torch.uint8):
        raise TypeError("done must be a torch.bool or torch.uint8 tensor")
    dense(done, "done", done.dtype, dev, (n,))
    dense(free_pages, "free_pages", torch.int32, dev)
    dense(free_count, "free_count", torch.int32, dev, (1,))
    return ctypes.byref(PageShape(n, width, 0, free_pages.shape.numel(), page))


def page_release(block_table, kv_lens, done, free_pages, free_count, page, stream=None):
    """Gives the pages of ended requests back (gdr_page_release): done [num_seqs] bool or uint8. The
    table, kv_lens, free_pages and free_count are changed in place."""
    lib = ops._load()
    shape = _checked_release(describe(block_table, "block_table"), describe(kv_lens, "kv_lens"), describe(done, "done"),
                             describe(free_pages, "free_pages"), describe(free_count, "free_count"), int(page))
    _launch(lib.gdr_page_release, "gdr_page_release", kv_lens.device, stream, shape, done.data_ptr(), kv_lens.data_ptr(),
            block_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr())


def _cache_fields(k_cache, v_cache, k_scale, v_scale, device, dtype):
    """The fields of CacheShape."""
    if k_cache.dtype not in _CODES:
        raise TypeError(f"unsupported k_cache: {k_cache.dtype}; torch.float8_e4m3fn or torch.int8")
    dense(k_cache, "k_cache", None, device)
    if len(k_cache.shape) != 4:
        raise ValueError("k_cache must have shape [num_pages, kv_heads, page, d]")
    shape = k_cache.shape
    dense(v_cache, "v_cache", k_cache.dtype, device, shape)
    dense(k_scale, "k_scale", torch.float32, device, shape[:2])
    dense(v_scale, "v_scale", torch.float32, device, shape[:2])
    pages, heads, page, d = shape
    return pages, heads, page, d, _CODES[k_cache.dtype], _DTYPES[dtype]


@functools.lru_cache(maxsize=256)
def _checked_append(k, v, slots, *caches):
    k, v, slots, *caches = named(k, v, slots, *caches)
    if k.dtype not in _DTYPES or len(k.shape) != 3:
        raise TypeError(f"unsupported k: {k.dtype}, {len(k.shape)} dimensions")
    dev, T = k.device, k.shape[0]
    ks, vs = rows_stride(k, "k", k.dtype, dev, T), rows_stride(v, "v", k.dtype, dev, T)
    cache = _cache_fields(*caches, dev, k.dtype)
    for t, name in ((k, "k"), (v, "v")):
        if t.shape[1] != cache[1] or t.shape[2] != cache[3]:
            raise ValueError(f"{name} must have shape ({T}, {cache[1]}, {cache[3]}), got {tuple(t.shape)}")
    dense(slots, "slots", torch.int32, dev, (T,))
    return ctypes.byref(CacheShape(*cache)), ks, vs


def cache_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream=None):
    """Puts new keys and values k, v [T, kv_heads, d] (bf16 or fp32, token strides of their own) into
    their slots [T] int32 (gdr_cache_append); rows with slot -1 are skipped. The caches and scales are
    changed in place."""
    lib = ops._load()
    shape, ks, vs = _checked_append(
        describe(k, "k"), describe(v, "v"), describe(slots, "slots"), describe(k_cache, "k_cache"),
        describe(v_cache, "v_cache"), describe(k_scale, "k_scale"), describe(v_scale, "v_scale"))
    _launch(lib.gdr_cache_append, "gdr_cache_append", k.device, stream, shape, k.shape[0], k.data_ptr(), ks, v.data_ptr(), vs,
            slots.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())


@functools.lru_cache(maxsize=256)
def _attn_call(cache, fields):
    """A reference to the struct of these fields, and the workspace bytes that it takes."""
    shape = ctypes.byref(CacheAttnShape(CacheShape(*cache), *fields))
    return shape, int(ops._load().gdr_cache_attn_workspace_size(shape))


def cache_attn_workspace_size(num_seqs, total_tokens, heads, kv_heads, d, page, width, num_pages, max_q=None,
                              dtype=torch.bfloat16, codes=torch.float8_e4m3fn):
    """Workspace bytes of cache_attn (0 if the sizes are unsupported)."""
    if max_q is None:
        max_q = total_tokens
    return _attn_call((int(num_pages), kv_heads, page, d, _CODES[codes], _DTYPES[dtype]),
                      (int(num_seqs), int(total_tokens), int(max_q), int(width), 0, heads, 1, 1.0, 0.0))[1]


@functools.lru_cache(maxsize=256)
def _checked_attn(q, caches, block_table, kv_lens, cu_q, slopes, o, lse, max_q, scale, softcap, causal):
    q, block_table, kv_lens, cu_q, slopes, o, lse = named(q, block_table, kv_lens, cu_q, slopes, o, lse)
    caches = named(*caches)
    if q.dtype not in _DTYPES or len(q.shape) != 3:
        raise TypeError(f"unsupported q: {q.dtype}, {len(q.shape)} dimensions")
    dev, dtype, (T, heads, d) = q.device, q.dtype, q.shape
    qs = rows_stride(q, "q", dtype, dev, T)
    cache = _cache_fields(*caches, dev, dtype)
    if cache[3] != d:
        raise ValueError(f"q has heads of {d}, the cache of {cache[3]}")
    _, n, width = _table(block_table)
    dense(block_table, "block_table", None, dev)
    dense(kv_lens, "kv_lens", torch.int32, dev, (n,))
    if cu_q is not None:
        dense(cu_q, "cu_q", torch.int32, dev, (n + 1,))
    if slopes is not None:
        dense(slopes, "slopes", torch.float32, dev, (heads,))
    if o is not None:
        dense(o, "o", dtype, dev, q.shape)
    if lse is not None:
        dense(lse, "lse", torch.float32, dev, (T, heads))
    if cu_q is None and n:
        max_q = T // n  # (T that n does not divide is refused)
    return _attn_call(cache, (n, T, T if max_q is None else max_q, width, qs, heads, causal, d ** -0.5 if scale is None else scale,
                              softcap))


def cache_attn(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_q=None, max_q=None, scale=None,
               softcap=0.0, slopes=None, causal=True, return_lse=False, o=None, lse=None, workspace=None, stream=None):
    """Softmax attention of the new tokens q [T, heads, d] over the cache (gdr_cache_attn), the
    new ones among the kv_lens [num_seqs] cached tokens of each request. cu_q [num_seqs + 1] int32:
    offsets of the requests' new tokens (max_q: the most of one request, default T; it chooses the kernel, so
    give 1 with the offsets of single tokens), or None for T / num_seqs each. Lengths that do not hold
    (kv_lens beyond the table, a request longer than max_q, ..) are found on the device: o and lse are then left
    as they were, which is unwritten memory if they are new, and read_device_status(workspace) of a
    workspace given by the caller tells. Prompts are planned by the table's width: a table about as wide
    as the lengths need is fastest and takes the least workspace. scale: default d^-1/2; softcap: scores capped by softcap tanh(s / softcap), 0 for none;
    slopes [heads] fp32: scores lowered by slope times the distance. Returns o [T, heads, d], with
    return_lse (o, lse [T, heads] fp32)."""
    lib = ops._load()
    shape, bytes_ = _checked_attn(
        describe(q, "q"), (describe(k_cache, "k_cache"), describe(v_cache, "v_cache"), describe(k_scale, "k_scale"),
                           describe(v_scale, "v_scale")),
        describe(block_table, "block_table"), describe(kv_lens, "kv_lens"), _opt(cu_q, "cu_q"), _opt(slopes, "slopes"),
        _opt(o, "o"), _opt(lse, "lse"), None if max_q is None else int(max_q), None if scale is None else float(scale),
        float(softcap), int(bool(causal)))
    if o is None:
        o = new_like(q, stream)
    if return_lse and lse is None:
        lse = new_like(q, stream, q.shape[:2], torch.float32)
    if workspace is None:
        workspace = new_like(q, stream, (max(bytes_, 256),), torch.uint8)
    else:
        _need(workspace, "workspace", device=q.device)
        bytes_ = workspace.nbytes
    _launch(lib.gdr_cache_attn, "gdr_cache_attn", q.device, stream, shape, q.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr(),
            _addr(cu_q), _addr(slopes), o.data_ptr(), _addr(lse), workspace.data_ptr(), bytes_)
    return (o, lse) if return_lse else o
