"""Rotary positions of queries and keys: binding of gdr_rotary_* (gdr.h).

The first rot_dim entries of a head are pairs, turned by an angle that grows with the token's
position; rates[i] is the turn of pair i per position in steps of 2^-64 of a whole one. q and k are
[T, heads, d] in bf16 or fp32 and may be views with a token stride of their own. Argument
marshalling only: there is no autograd here, `rotary_bwd` turns gradients back.
"""
import ctypes
import functools
import math

import torch

from . import ops
from .linattn import _addr, _new, _rows
from .ops import _DTYPES, _launch, _need


class RotaryShape(ctypes.Structure):
    """struct gdr_rotary_shape of gdr.h."""
    _fields_ = [("tokens", ctypes.c_int64), ("q_heads", ctypes.c_int), ("k_heads", ctypes.c_int),
                ("d", ctypes.c_int), ("rot_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("neighbours", ctypes.c_int), ("amplitude", ctypes.c_float),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64)]


@functools.lru_cache(maxsize=256)
def _shape(fields):
    """A reference to the struct of these fields."""
    return ctypes.byref(RotaryShape(*fields))


def rotary_rates(rot_dim, base=10000.0, factor=1.0, trained_length=None, fast_turns=32.0, slow_turns=1.0,
                 device="cuda"):
    """The rates of rot_dim / 2 pairs, int64: pair i turns by base^(-2i / rot_dim) radians per
    position, in 64 bits, to the nearest 2^-64 of a turn.

    factor > 1 stretches the context: without trained_length every pair turns `factor` times
    slower (positions interpolated). With it, pairs that turn more than fast_turns times within
    trained_length positions keep their rate, those of less than slow_turns are slowed by
    factor, with a ramp between them (interpolation by parts; rotary_amplitude goes with it)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and positive, got {rot_dim}")
    if not (math.isfinite(base) and base > 0 and math.isfinite(factor) and factor > 0):
        raise ValueError("base and factor must be positive and finite")
    if trained_length is not None and not fast_turns > slow_turns:
        raise ValueError("fast_turns must be above slow_turns")
    rates = []
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        keep = 0.0
        if trained_length is not None:
            turns = trained_length * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - slow_turns) / (fast_turns - slow_turns)))
        f = f * keep + f / factor * (1 - keep)
        r = round(f / (2 * math.pi) * 2.0 ** 64) % 2 ** 64
        rates.append(r - 2 ** 64 if r >= 2 ** 63 else r)
    return torch.tensor(rates, dtype=torch.int64, device=device)


def rotary_amplitude(factor):
    """The amplitude that goes with interpolation by parts: 0.1 ln(factor) + 1 (1 up to a factor of 1)."""
    return 1.0 if factor <= 1 else 0.1 * math.log(factor) + 1.0


def _out(t, name, like, stream):
    """A given output of `like`'s shape and its token stride, or a new dense one."""
    if t is None:
        return _new(like.shape, like.dtype, like.device, stream), 0
    stride = _rows(t, name, like.dtype, like.device, like.shape[0])
    if t.shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
    return t, stride


def _rotary(f, what, names, q, k, positions, rates, neighbours, amplitude, q_out, k_out, stream):
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES or q.dim() != 3:
        raise TypeError(f"unsupported {names[0]}: {getattr(q, 'dtype', type(q))}")
    dev, dtype, (T, q_heads, d) = q.device, q.dtype, q.shape
    qs = _rows(q, names[0], dtype, dev, T)
    ks, k_heads = 0, 0
    if k is not None:
        ks = _rows(k, names[1], dtype, dev, T)
        k_heads = k.shape[1]
        if k.shape[2] != d:
            raise ValueError(f"{names[1]} has heads of {k.shape[2]}, {names[0]} of {d}")
    _need(positions, "positions", torch.int32, dev)
    _need(rates, "rates", torch.int64, dev)
    if positions.dim() != 1 or positions.shape[0] != T:
        raise ValueError(f"positions must have shape ({T},), got {tuple(positions.shape)}")
    if rates.dim() != 1:
        raise ValueError("rates must have shape [rot_dim / 2]")
    q_out, qos = _out(q_out, names[2], q, stream)
    kos = 0
    if k is not None:
        k_out, kos = _out(k_out, names[3], k, stream)
    elif k_out is not None:
        raise ValueError(f"{names[3]} needs {names[1]}")
    _launch(f, what, dev, stream,
            _shape((T, q_heads, k_heads, d, 2 * rates.shape[0], _DTYPES[dtype], int(bool(neighbours)), float(amplitude),
                    qs, ks, qos, kos)),
            q.data_ptr(), _addr(k), positions.data_ptr(), rates.data_ptr(), q_out.data_ptr(), _addr(k_out))
    return q_out, k_out


def rotary_fwd(q, k, positions, rates, neighbours=False, amplitude=1.0, q_out=None, k_out=None, stream=None):
    """Queries q [T, q_heads, d] and keys k [T, k_heads, d] (or None) turned to their positions
    [T] int32 (gdr_rotary_fwd). A pair is entries i and i + rot_dim / 2, with `neighbours` 2i and 2i + 1;
    rot_dim = 2 len(rates) may be less than d. Returns (q_out, k_out): new tensors, or those
    given; q_out may be q and k_out may be k."""
    return _rotary(ops._load().gdr_rotary_fwd, "gdr_rotary_fwd", ("q", "k", "q_out", "k_out"), q, k, positions, rates,
                   neighbours, amplitude, q_out, k_out, stream)


def rotary_bwd(dq_out, dk_out, positions, rates, neighbours=False, amplitude=1.0, dq=None, dk=None, stream=None):
    """Gradients of rotary_fwd's q and k from those of its outputs (gdr_rotary_bwd): the turn
    back. Returns (dq, dk); dq may be dq_out and dk may be dk_out."""
    return _rotary(ops._load().gdr_rotary_bwd, "gdr_rotary_bwd", ("dq_out", "dk_out", "dq", "dk"), dq_out, dk_out,
                   positions, rates, neighbours, amplitude, dq, dk, stream)
