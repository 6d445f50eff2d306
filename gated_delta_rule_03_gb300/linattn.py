"""Linear attention with one constant decay per head: binding of gdr_linattn_* (gdr.h).

S_t = lam S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t with lam = exp(log_decay[h]). q, k and v
are [T, heads, d] in bf16 or fp32, each with a head count that divides H (the length of
log_decay). They may be views with a token stride of their own, as the parts of one fused
projection are; everything else is dense. Argument marshalling only: there is no autograd
here, `linattn_bwd` returns the gradients.
"""
import ctypes
import functools

import torch

from . import ops
from .ops import _DTYPES, _launch, _need


class LinattnShape(ctypes.Structure):
    """struct gdr_linattn_shape of gdr.h."""
    _fields_ = [("num_seqs", ctypes.c_int64), ("total_tokens", ctypes.c_int64),
                ("H", ctypes.c_int), ("q_heads", ctypes.c_int), ("k_heads", ctypes.c_int),
                ("v_heads", ctypes.c_int), ("d_k", ctypes.c_int), ("d_v", ctypes.c_int),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64)]


@functools.lru_cache(maxsize=256)
def _shape(fields):
    """A reference to the struct of these fields."""
    return ctypes.byref(LinattnShape(*fields))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(backward, fields):
    lib = ops._load()
    f = lib.gdr_linattn_bwd_workspace_size if backward else lib.gdr_linattn_fwd_workspace_size
    return int(f(_shape(fields)))


def _rows(t, name, dtype, device, tokens):
    """Checks a [tokens, heads, d] tensor whose heads are contiguous; its token stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have shape [tokens, heads, d]")
    n, heads, d = t.shape
    if n != tokens:
        raise ValueError(f"{name} has {n} tokens, expected {tokens}")
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (heads > 1 and s1 != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if n <= 1:
        return heads * d
    if s0 < heads * d:
        raise ValueError(f"{name}: the token stride must be at least heads * d")
    return s0


def _fields(q, k, v, log_decay, n, scale):
    """The fields of LinattnShape; n: sequences, None for one per token."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES:
        raise TypeError(f"unsupported q: {getattr(q, 'dtype', type(q))}")
    dtype, device = q.dtype, q.device
    T = q.shape[0] if q.dim() else 0
    qs = _rows(q, "q", dtype, device, T)
    ks = _rows(k, "k", dtype, device, T)
    vs = _rows(v, "v", dtype, device, T)
    _, q_heads, d_k = q.shape
    _, k_heads, d = k.shape
    _, v_heads, d_v = v.shape
    if d != d_k:
        raise ValueError(f"k has heads of {d}, q of {d_k}")
    _need(log_decay, "log_decay", torch.float32, device)
    if log_decay.dim() != 1:
        raise ValueError("log_decay must have shape [H]")
    return (T if n is None else n, T, log_decay.numel(), q_heads, k_heads, v_heads, d_k, d_v, _DTYPES[dtype], float(scale), qs, ks, vs)


def _seqs(cu_seqlens, num_seqs, device):
    if cu_seqlens is None:
        return 1 if num_seqs is None else int(num_seqs)
    _need(cu_seqlens, "cu_seqlens", torch.int32, device)
    n = cu_seqlens.numel() - 1
    if num_seqs is not None and int(num_seqs) != n:
        raise ValueError(f"num_seqs is {num_seqs}, cu_seqlens has {n} sequences")
    return n


def _new(shape, dtype, device, stream):
    """A tensor to be written on `stream`: memory of that stream, so that what the current
    stream still does with memory it has given back does not run into it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _dense(t, name, shape, dtype, device, stream=None):
    """A given output, checked, or a new one."""
    if t is None:
        return _new(shape, dtype, device, stream)
    _need(t, name, dtype, device)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _given(t, name, shape, dtype, device):
    if t is not None:
        _dense(t, name, shape, dtype, device)


def _addr(t):
    return None if t is None else t.data_ptr()


def linattn_fwd_workspace_size(num_seqs, total_tokens, H, dk, dv, dtype=torch.bfloat16,
                               q_heads=None, k_heads=None, v_heads=None):
    """Workspace bytes of linattn_fwd (0 if the sizes are unsupported)."""
    return _workspace_bytes(False, (int(num_seqs), int(total_tokens), H, q_heads or H, k_heads or H,
                            v_heads or H, dk, dv, _DTYPES[dtype], 1.0, 0, 0, 0))


def linattn_bwd_workspace_size(num_seqs, total_tokens, H, dk, dv, dtype=torch.bfloat16,
                               q_heads=None, k_heads=None, v_heads=None):
    """Workspace bytes of linattn_bwd (0 if the sizes are unsupported)."""
    return _workspace_bytes(True, (int(num_seqs), int(total_tokens), H, q_heads or H, k_heads or H,
                            v_heads or H, dk, dv, _DTYPES[dtype], 1.0, 0, 0, 0))


def _workspace(workspace, backward, fields, device, stream):
    if workspace is None:
        return _new(max(_workspace_bytes(backward, fields), 256), torch.uint8, device, stream)
    _need(workspace, "workspace", device=device)
    return workspace


def linattn_fwd(q, k, v, log_decay, S0=None, cu_seqlens=None, num_seqs=None, scale=1.0,
                final_state=True, o=None, S_final=None, workspace=None, stream=None):
    """Prompts (gdr_linattn_fwd): q [T, q_heads, dk], k [T, k_heads, dk], v [T, v_heads, dv];
    log_decay [H] fp32; S0 [num_seqs, H, dk, dv] fp32 or None; cu_seqlens [num_seqs + 1]
    int32 or None (then `num_seqs` equal sequences, default 1). Returns (o [T, H, dv],
    S_final [num_seqs, H, dk, dv] fp32, or None with final_state=False). Preallocated o,
    S_final (which may be S0) and workspace (uint8) are used as given."""
    lib = ops._load()
    n = _seqs(cu_seqlens, num_seqs, q.device)
    fields = _fields(q, k, v, log_decay, n, scale)
    dev, (T, H, dk, dv) = q.device, (fields[1], fields[2], fields[6], fields[7])
    _given(S0, "S0", (n, H, dk, dv), torch.float32, dev)
    o = _dense(o, "o", (T, H, dv), q.dtype, dev, stream)
    if final_state or S_final is not None:
        S_final = _dense(S_final, "S_final", (n, H, dk, dv), torch.float32, dev, stream)
    ws = _workspace(workspace, False, fields, dev, stream)
    _launch(lib.gdr_linattn_fwd, "gdr_linattn_fwd", dev, stream, _shape(fields), q.data_ptr(), k.data_ptr(),
            v.data_ptr(), log_decay.data_ptr(), _addr(S0), _addr(cu_seqlens), o.data_ptr(), _addr(S_final),
            ws.data_ptr(), ws.nbytes)
    return o, S_final


def linattn_bwd(do, q, k, v, log_decay, S0=None, dS_final=None, cu_seqlens=None, num_seqs=None,
                scale=1.0, dq=None, dk=None, dv=None, dS0=None, workspace=None, stream=None):
    """Gradients of linattn_fwd (gdr_linattn_bwd) from do [T, H, dv] and the gradient
    dS_final of S_final (None for zero). Returns (dq, dk, dv, dS0), each like its tensor but
    dense; dS0 is None unless S0 or dS0 is given."""
    lib = ops._load()
    n = _seqs(cu_seqlens, num_seqs, q.device)
    fields = _fields(q, k, v, log_decay, n, scale)
    dev, (T, H, d_k, d_v) = q.device, (fields[1], fields[2], fields[6], fields[7])
    state = (n, H, d_k, d_v)
    _given(S0, "S0", state, torch.float32, dev)
    _given(dS_final, "dS_final", state, torch.float32, dev)
    if do is None:
        raise TypeError("do must be a torch.Tensor")
    _given(do, "do", (T, H, d_v), q.dtype, dev)
    dq = _dense(dq, "dq", q.shape, q.dtype, dev, stream)
    dk = _dense(dk, "dk", k.shape, q.dtype, dev, stream)
    dv = _dense(dv, "dv", v.shape, q.dtype, dev, stream)
    if S0 is not None or dS0 is not None:
        dS0 = _dense(dS0, "dS0", state, torch.float32, dev, stream)
    ws = _workspace(workspace, True, fields, dev, stream)
    _launch(lib.gdr_linattn_bwd, "gdr_linattn_bwd", dev, stream, _shape(fields), do.data_ptr(), q.data_ptr(),
            k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _addr(S0), _addr(dS_final), _addr(cu_seqlens),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _addr(dS0), ws.data_ptr(), ws.nbytes)
    return dq, dk, dv, dS0


def linattn_step(q, k, v, log_decay, S, scale=1.0, o=None, stream=None):
    """The next token of N sequences (gdr_linattn_step): q [N, q_heads, dk], k [N, k_heads,
    dk], v [N, v_heads, dv]; S [N, H, dk, dv] fp32 updated in place. Returns o [N, H, dv]."""
    lib = ops._load()
    fields = _fields(q, k, v, log_decay, None, scale)
    dev, (N, H, dk, dv) = q.device, (fields[1], fields[2], fields[6], fields[7])
    if S is None:
        raise TypeError("S must be a torch.Tensor")
    _given(S, "S", (N, H, dk, dv), torch.float32, dev)
    o = _dense(o, "o", (N, H, dv), q.dtype, dev, stream)
    _launch(lib.gdr_linattn_step, "gdr_linattn_step", dev, stream, _shape(fields), q.data_ptr(), k.data_ptr(),
            v.data_ptr(), log_decay.data_ptr(), S.data_ptr(), o.data_ptr())
    return o
