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
from .linattn import _addr, _dense, _new, _rows
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


@functools.lru_cache(maxsize=256)
def _page_shape(fields):
    return ctypes.byref(PageShape(*fields))


@functools.lru_cache(maxsize=256)
def _cache_shape(fields):
    return ctypes.byref(CacheShape(*fields))


@functools.lru_cache(maxsize=256)
def _attn_shape(cache, fields):
    return ctypes.byref(CacheAttnShape(CacheShape(*cache), *fields))


@functools.lru_cache(maxsize=256)
def _attn_workspace_bytes(cache, fields):
    return int(ops._load().gdr_cache_attn_workspace_size(_attn_shape(cache, fields)))


def _table(block_table):
    _need(block_table, "block_table", torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must have shape [num_seqs, width]")
    return block_table.device, block_table.shape[0], block_table.shape[1]


def _vector(t, name, n, dtype, device):
    _need(t, name, dtype, device)
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must have shape ({n},), got {tuple(t.shape)}")
    return t


def page_plan(block_table, kv_lens, free_pages, free_count, page, q_lens=None, rows=None, kv_lens_out=None,
              free_count_out=None, cu_q=None, start=None, positions=None, slots=None, stream=None):
    """Pages, positions and slots of the requests' new tokens (gdr_page_plan): block_table
    [num_seqs, width], kv_lens [num_seqs], free_pages [num_pages] and free_count [1] int32; q_lens
    [num_seqs] int32 or None for one token each; rows: tokens of the packed batch, padding included
    (default num_seqs; needed with q_lens). The table gets its new entries in place. Returns a
    PagePlan (kv_lens, free_count, cu_q, start, positions, slots) of new tensors or those given; kv_lens_out
    may be kv_lens and free_count_out may be free_count. start is -1 for a refused request."""
    lib = ops._load()
    dev, n, width = _table(block_table)
    _vector(kv_lens, "kv_lens", n, torch.int32, dev)
    _need(free_pages, "free_pages", torch.int32, dev)
    _vector(free_count, "free_count", 1, torch.int32, dev)
    if q_lens is not None:
        _vector(q_lens, "q_lens", n, torch.int32, dev)
        if rows is None:
            raise ValueError("q_lens needs rows, the tokens of the packed batch")
    rows = n if rows is None else int(rows)
    i32 = torch.int32
    kv_lens_out = _dense(kv_lens_out, "kv_lens_out", (n,), i32, dev, stream)
    free_count_out = _dense(free_count_out, "free_count_out", (1,), i32, dev, stream)
    cu_q = _dense(cu_q, "cu_q", (n + 1,), i32, dev, stream)
    start = _dense(start, "start", (n,), i32, dev, stream)
    positions = _dense(positions, "positions", (rows,), i32, dev, stream)
    slots = _dense(slots, "slots", (rows,), i32, dev, stream)
    _launch(lib.gdr_page_plan, "gdr_page_plan", dev, stream, _page_shape((n, width, rows, free_pages.numel(), int(page))),
            _addr(q_lens), kv_lens.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), block_table.data_ptr(),
            kv_lens_out.data_ptr(), free_count_out.data_ptr(), cu_q.data_ptr(), start.data_ptr(), positions.data_ptr(),
            slots.data_ptr())
    return PagePlan(kv_lens_out, free_count_out, cu_q, start, positions, slots)


def page_release(block_table, kv_lens, done, free_pages, free_count, page, stream=None):
    """Gives the pages of ended requests back (gdr_page_release): done [num_seqs] bool or uint8. The
    table, kv_lens, free_pages and free_count are changed in place."""
    lib = ops._load()
    dev, n, width = _table(block_table)
    _vector(kv_lens, "kv_lens", n, torch.int32, dev)
    if not isinstance(done, torch.Tensor) or done.dtype not in (torch.bool, torch.uint8):
        raise TypeError("done must be a torch.bool or torch.uint8 tensor")
    _vector(done, "done", n, done.dtype, dev)
    _need(free_pages, "free_pages", torch.int32, dev)
    _vector(free_count, "free_count", 1, torch.int32, dev)
    _launch(lib.gdr_page_release, "gdr_page_release", dev, stream, _page_shape((n, width, 0, free_pages.numel(), int(page))),
            done.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr())


def _cache(k_cache, v_cache, k_scale, v_scale, device, dtype):
    """The fields of CacheShape."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dtype not in _CODES:
        raise TypeError(f"unsupported k_cache: {getattr(k_cache, 'dtype', type(k_cache))}; torch.float8_e4m3fn or torch.int8")
    _need(k_cache, "k_cache", None, device)
    if k_cache.dim() != 4:
        raise ValueError("k_cache must have shape [num_pages, kv_heads, page, d]")
    shape = k_cache.shape
    for t, name, want, of in ((v_cache, "v_cache", shape, k_cache.dtype), (k_scale, "k_scale", shape[:2], torch.float32),
                              (v_scale, "v_scale", shape[:2], torch.float32)):
        _need(t, name, of, device)
        if t.shape != want:
            raise ValueError(f"{name} must have shape {tuple(want)}, got {tuple(t.shape)}")
    pages, heads, page, d = shape
    return pages, heads, page, d, _CODES[k_cache.dtype], _DTYPES[dtype]


def cache_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream=None):
    """Puts new keys and values k, v [T, kv_heads, d] (bf16 or fp32, token strides of their own) into
    their slots [T] int32 (gdr_cache_append); rows with slot -1 are skipped. The caches and scales are
    changed in place."""
    lib = ops._load()
    if not isinstance(k, torch.Tensor) or k.dtype not in _DTYPES or k.dim() != 3:
        raise TypeError(f"unsupported k: {getattr(k, 'dtype', type(k))}")
    dev, T = k.device, k.shape[0]
    ks, vs = _rows(k, "k", k.dtype, dev, T), _rows(v, "v", k.dtype, dev, T)
    cache = _cache(k_cache, v_cache, k_scale, v_scale, dev, k.dtype)
    for t, name in ((k, "k"), (v, "v")):
        if t.shape[1] != cache[1] or t.shape[2] != cache[3]:
            raise ValueError(f"{name} must have shape ({T}, {cache[1]}, {cache[3]}), got {tuple(t.shape)}")
    _vector(slots, "slots", T, torch.int32, dev)
    _launch(lib.gdr_cache_append, "gdr_cache_append", dev, stream, _cache_shape(cache), T, k.data_ptr(), ks, v.data_ptr(),
            vs, slots.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())


def cache_attn_workspace_size(num_seqs, total_tokens, heads, kv_heads, d, page, width, num_pages, max_q=None,
                              dtype=torch.bfloat16, codes=torch.float8_e4m3fn):
    """Workspace bytes of cache_attn (0 if the sizes are unsupported)."""
    if max_q is None:
        max_q = total_tokens
    return _attn_workspace_bytes((int(num_pages), kv_heads, page, d, _CODES[codes], _DTYPES[dtype]),
                                 (int(num_seqs), int(total_tokens), int(max_q), int(width), 0, heads, 1, 1.0, 0.0))


def cache_attn(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_q=None, max_q=None, scale=None,
               softcap=0.0, slopes=None, causal=True, return_lse=False, o=None, lse=None, workspace=None, stream=None):
    """Softmax attention of the new tokens q [T, heads, d] over the cache (gdr_cache_attn), the
    new ones among the kv_lens [num_seqs] cached tokens of each request. cu_q [num_seqs + 1] int32:
    offsets of the requests' new tokens (max_q: the most of one request, default T), or None for T /
    num_seqs each. scale: default d^-1/2; softcap: scores capped by softcap tanh(s / softcap), 0 for none;
    slopes [heads] fp32: scores lowered by slope times the distance. Returns o [T, heads, d], with
    return_lse (o, lse [T, heads] fp32)."""
    lib = ops._load()
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES or q.dim() != 3:
        raise TypeError(f"unsupported q: {getattr(q, 'dtype', type(q))}")
    dev, dtype, (T, heads, d) = q.device, q.dtype, q.shape
    qs = _rows(q, "q", dtype, dev, T)
    cache = _cache(k_cache, v_cache, k_scale, v_scale, dev, dtype)
    if cache[3] != d:
        raise ValueError(f"q has heads of {d}, the cache of {cache[3]}")
    _need(block_table, "block_table", torch.int32, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must have shape [num_seqs, width]")
    n, width = block_table.shape
    _vector(kv_lens, "kv_lens", n, torch.int32, dev)
    if cu_q is not None:
        _vector(cu_q, "cu_q", n + 1, torch.int32, dev)
    if slopes is not None:
        _vector(slopes, "slopes", heads, torch.float32, dev)
    fields = (n, T, T if max_q is None else int(max_q), width, qs, heads, int(bool(causal)),
              d ** -0.5 if scale is None else float(scale), float(softcap))
    o = _dense(o, "o", q.shape, dtype, dev, stream)
    if return_lse or lse is not None:
        lse = _dense(lse, "lse", (T, heads), torch.float32, dev, stream)
    if workspace is None:
        workspace = _new(max(_attn_workspace_bytes(cache, fields), 256), torch.uint8, dev, stream)
    _need(workspace, "workspace", device=dev)
    _launch(lib.gdr_cache_attn, "gdr_cache_attn", dev, stream, _attn_shape(cache, fields), q.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr(),
            _addr(cu_q), _addr(slopes), o.data_ptr(), _addr(lse), workspace.data_ptr(), workspace.nbytes)
    return (o, lse) if return_lse else o
