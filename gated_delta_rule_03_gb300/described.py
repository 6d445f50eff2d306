"""Checks of tensors by what can be said of them without their data.

`describe` takes a tensor's type, shape, strides and device; the checks of a call take only such
descriptions, so that a call whose tensors look like those of an earlier one finds its result in a cache
(a dozen checks take 10 us of a small call).
"""
import collections

import torch

empty = torch.empty
Described = collections.namedtuple("Described", "dtype shape stride device")


def describe(t, name):
    """A plain tuple, half the time of the named one, which `named` makes of it."""
    try:
        return t.dtype, t.shape, t.stride(), t.device
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None


def named(*descriptions):
    return [t if t is None else Described(*t) for t in descriptions]


def _contiguous(t):
    expected = 1
    for n, s in zip(reversed(t.shape), reversed(t.stride)):
        if n == 0:
            return True
        if n != 1:
            if s != expected:
                return False
            expected *= n
    return True


def dense(t, name, dtype=None, device=None, shape=None):
    """A contiguous CUDA tensor of this type, device and shape (where given)."""
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if not _contiguous(t):
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def rows_stride(t, name, dtype, device, tokens):
    """The token stride of a [tokens, heads, d] tensor whose heads are contiguous."""
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if len(t.shape) != 3:
        raise ValueError(f"{name} must have shape [tokens, heads, d]")
    n, heads, d = t.shape
    if n != tokens:
        raise ValueError(f"{name} has {n} tokens, expected {tokens}")
    s0, s1, s2 = t.stride
    if (d > 1 and s2 != 1) or (heads > 1 and s1 != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if n <= 1:
        return heads * d
    if s0 < heads * d:
        raise ValueError(f"{name}: the token stride must be at least heads * d")
    return s0


def new_like(t, stream, shape=None, dtype=None):
    """A dense tensor to be written on `stream`: memory of that stream."""
    if stream is None:
        return empty(t.shape if shape is None else shape, dtype=dtype or t.dtype, device=t.device)
    with torch.cuda.stream(stream):
        return empty(t.shape if shape is None else shape, dtype=dtype or t.dtype, device=t.device)
