"""Rotary positions of queries and keys: binding of gdr_rotary_* (gdr.h).

The first rot_dim entries of a head are pairs, turned by an angle that grows with the token's
position; rates[i] is the turn of pair i per position in steps of 2^-64 of a whole one. q and k are
[T, heads, d] in bf16 or fp32 and may be views with a token stride of their own. Argument
marshalling only: there is no autograd here, `rotary_bwd` turns gradients back.
"""
import ctypes
import decimal
import functools
import math

import torch

from . import ops
from .described import dense, describe, named, new_like, rows_stride
from .linattn import _addr
from .ops import _DTYPES, _launch


class RotaryShape(ctypes.Structure):
    """struct gdr_rotary_shape of gdr.h."""
    _fields_ = [("tokens", ctypes.c_int64), ("q_heads", ctypes.c_int), ("k_heads", ctypes.c_int),
                ("d", ctypes.c_int), ("rot_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("neighbours", ctypes.c_int), ("amplitude", ctypes.c_float),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64)]


_TWO_PI = decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194989")


def rotary_rates(rot_dim, base=10000.0, factor=1.0, trained_length=None, fast_turns=32.0, slow_turns=1.0,
                 device="cuda"):
    """The rates of rot_dim / 2 pairs, int64: pair i turns by base^(-2i / rot_dim) radians per
    position, to the nearest 2^-64 of a turn (in decimals: doubles would leave 2^-56 of the fastest pairs).

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
    with decimal.localcontext(decimal.Context(prec=50)):
        base, factor, lo, hi = (decimal.Decimal(float(x)) for x in (base, factor, slow_turns, fast_turns))
        for i in range(rot_dim // 2):
            turns = base ** (decimal.Decimal(-2 * i) / int(rot_dim)) / _TWO_PI
            keep = 0
            if trained_length is not None:
                keep = min(1, max(0, (decimal.Decimal(float(trained_length)) * turns - lo) / (hi - lo)))
            turns = turns * keep + turns / factor * (1 - keep)
            r = int((turns * 2 ** 64).to_integral_value(decimal.ROUND_HALF_EVEN)) % 2 ** 64
            rates.append(r - 2 ** 64 if r >= 2 ** 63 else r)
    return torch.tensor(rates, dtype=torch.int64, device=device)


def rotary_amplitude(factor):
    """The amplitude that goes with interpolation by parts: 0.1 ln(factor) + 1 (1 up to a factor of 1)."""
    return 1.0 if factor <= 1 else 0.1 * math.log(factor) + 1.0


@functools.lru_cache(maxsize=256)
def _checked(names, q, k, positions, rates, q_out, k_out, neighbours, amplitude):
    """Checks tensors by what `describe` says of them; a reference to the struct of the call."""
    q, k, positions, rates, q_out, k_out = named(q, k, positions, rates, q_out, k_out)
    if q.dtype not in _DTYPES or len(q.shape) != 3:
        raise TypeError(f"unsupported {names[0]}: {q.dtype}, {len(q.shape)} dimensions")
    dev, dtype, (T, q_heads, d) = q.device, q.dtype, q.shape
    qs = rows_stride(q, names[0], dtype, dev, T)
    ks, kos, k_heads = 0, 0, 0
    if k is not None:
        ks = rows_stride(k, names[1], dtype, dev, T)
        k_heads = k.shape[1]
        if k.shape[2] != d:
            raise ValueError(f"{names[1]} has heads of {k.shape[2]}, {names[0]} of {d}")
    dense(positions, "positions", torch.int32, dev, (T,))
    dense(rates, "rates", torch.int64, dev)
    if len(rates.shape) != 1:
        raise ValueError("rates must have shape [rot_dim / 2]")

    def out_stride(t, name, like):
        if t is None:
            return 0
        stride = rows_stride(t, name, dtype, dev, T)
        if t.shape != like.shape:
            raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
        return stride

    qos = out_stride(q_out, names[2], q)
    if k is not None:
        kos = out_stride(k_out, names[3], k)
    elif k_out is not None:
        raise ValueError(f"{names[3]} needs {names[1]}")
    return ctypes.byref(RotaryShape(T, q_heads, k_heads, d, 2 * rates.shape[0], _DTYPES[dtype], neighbours, amplitude, qs, ks,
                                    qos, kos))


def _rotary(f, what, names, q, k, positions, rates, neighbours, amplitude, q_out, k_out, stream):
    shape = _checked(names, describe(q, names[0]), k if k is None else describe(k, names[1]), describe(positions, "positions"),
                     describe(rates, "rates"), q_out if q_out is None else describe(q_out, names[2]),
                     k_out if k_out is None else describe(k_out, names[3]), int(bool(neighbours)), float(amplitude))
    if q_out is None:
        q_out = new_like(q, stream)
    if k is not None and k_out is None:
        k_out = new_like(k, stream)
    _launch(f, what, q.device, stream, shape, q.data_ptr(), _addr(k), positions.data_ptr(), rates.data_ptr(),
            q_out.data_ptr(), _addr(k_out))
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
