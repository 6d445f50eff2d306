"""The norms before and after a block with its gate and the residual scale: binding of
gdr_block_norm_* (gdr.h).

x' = x + res_scale act(gate) t with t = rmsnorm(y) w_post (post_norm; else y), and
h = rmsnorm(x') w_pre (pre_norm). Tensors are dense [..., D]; y, gate and h share a type, x
and x' have that type or fp32; weights are fp32. Argument marshalling only: there is no
autograd here, `block_norm_bwd` returns the gradients.
"""
import ctypes
import functools

import torch

from . import ops
from .linattn import _addr, _dense, _given, _new
from .ops import _DTYPES, _launch, _need

# the gate's function (gdr_block_norm_shape.gate_act)
ACTS = {"identity": 0, "silu": 1, "sigmoid": 2}


class BlockNormShape(ctypes.Structure):
    """struct gdr_block_norm_shape of gdr.h."""
    _fields_ = [("rows", ctypes.c_int64), ("D", ctypes.c_int), ("dtype", ctypes.c_int),
                ("x_dtype", ctypes.c_int), ("post_norm", ctypes.c_int), ("pre_norm", ctypes.c_int),
                ("gate_act", ctypes.c_int), ("gate_rows", ctypes.c_int64),
                ("res_scale", ctypes.c_float), ("eps", ctypes.c_float)]


@functools.lru_cache(maxsize=256)
def _shape(fields):
    """A reference to the struct of these fields."""
    return ctypes.byref(BlockNormShape(*fields))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(fields):
    return int(ops._load().gdr_block_norm_bwd_workspace_size(_shape(fields)))


def _fields(x, y, gate, act, w_post, w_pre, post_norm, pre_norm, res_scale, eps, dtype):
    _need(x, "x")
    if x.dim() < 1 or x.dtype not in _DTYPES:
        raise TypeError(f"unsupported x: {tuple(x.shape)} {x.dtype}")
    if act not in ACTS:
        raise ValueError(f"unknown act {act!r}; expected one of {sorted(ACTS)}")
    dev, D = x.device, x.shape[-1]
    rows = x.numel() // D if D else 0
    if y is not None:
        dtype = y.dtype
        _given(y, "y", x.shape, dtype, dev)
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    gate_rows = 0
    if gate is not None:
        _need(gate, "gate", dtype, dev)
        if gate.numel() == D and (gate.dim() < 2 or gate.shape[-1] == D):
            gate_rows = 1
        elif tuple(gate.shape) == tuple(x.shape):
            gate_rows = rows
        else:
            raise ValueError(f"gate must have shape {tuple(x.shape)} or one row of {D}")
    for name, w, used in (("w_post", w_post, post_norm), ("w_pre", w_pre, pre_norm)):
        if w is not None:
            if not used:
                raise ValueError(f"{name} needs its norm")
            _given(w, name, (D,), torch.float32, dev)
    return (rows, D, _DTYPES[dtype], _DTYPES[x.dtype], int(bool(post_norm)), int(bool(pre_norm)),
            ACTS[act], gate_rows, float(res_scale), float(eps))


def block_norm_fwd(x, y=None, gate=None, act="silu", w_post=None, w_pre=None, post_norm=True,
                   pre_norm=True, res_scale=1.0, eps=1e-6, dtype=None, x_out=None, h=None,
                   stream=None):
    """Returns (x', h): the residual stream behind the block and the next block's normed
    input (None without pre_norm). x_out may be x. gate: like y, or one row [D] for all.
    Without y, h = rmsnorm(x) w_pre in `dtype` (default x's), and x' is x itself."""
    lib = ops._load()
    if y is None:
        post_norm = False
    fields = _fields(x, y, gate, act, w_post, w_pre, post_norm, pre_norm, res_scale, eps, dtype or x.dtype)
    dev = x.device
    dt = y.dtype if y is not None else (dtype or x.dtype)
    if y is not None:
        x_out = _dense(x_out, "x_out", x.shape, x.dtype, dev, stream)
    elif x_out is not None:
        raise ValueError("x_out needs y")
    if pre_norm:
        h = _dense(h, "h", x.shape, dt, dev, stream)
    elif h is not None:
        raise ValueError("h needs pre_norm")
    _launch(lib.gdr_block_norm_fwd, "gdr_block_norm_fwd", dev, stream, _shape(fields), x.data_ptr(), _addr(y),
            _addr(gate), _addr(w_post), _addr(w_pre), _addr(x_out), _addr(h))
    return (x if y is None else x_out), h


def block_norm_bwd_workspace_size(rows, D, dtype=torch.bfloat16, x_dtype=None):
    """Workspace bytes of block_norm_bwd (0 if the sizes are unsupported)."""
    return _workspace_bytes((int(rows), int(D), _DTYPES[dtype], _DTYPES[x_dtype or dtype], 1, 1, 0, 0, 1.0, 0.0))


def block_norm_bwd(dx_out, dh, x_out, y=None, gate=None, act="silu", w_post=None, w_pre=None,
                   post_norm=True, pre_norm=True, res_scale=1.0, eps=1e-6, dx=None, dy=None,
                   dgate=None, dw_post=None, dw_pre=None, workspace=None, stream=None):
    """Gradients of block_norm_fwd from dh (with pre_norm) and dx_out, the gradient of x'
    from behind the block (None for zero, with pre_norm only). x_out is the stored x'.
    Returns (dx, dy, dgate, dw_post, dw_pre), None where there is no such input. dx may be
    dx_out."""
    lib = ops._load()
    if y is None:
        post_norm = False
    if not isinstance(x_out, torch.Tensor):
        raise TypeError("x_out must be a torch.Tensor")
    dtype = y.dtype if y is not None else (dh.dtype if dh is not None else x_out.dtype)
    fields = _fields(x_out, y, gate, act, w_post, w_pre, post_norm, pre_norm, res_scale, eps, dtype)
    dev, D = x_out.device, fields[1]
    _given(dx_out, "dx_out", x_out.shape, x_out.dtype, dev)
    if pre_norm:
        if dh is None:
            raise ValueError("pre_norm needs dh")
        _given(dh, "dh", x_out.shape, dtype, dev)
    elif dh is not None:
        raise ValueError("dh needs pre_norm")
    dx = _dense(dx, "dx", x_out.shape, x_out.dtype, dev, stream)
    if y is not None:
        dy = _dense(dy, "dy", y.shape, dtype, dev, stream)
    if gate is not None:
        dgate = _dense(dgate, "dgate", gate.shape, dtype, dev, stream)
    if w_post is not None:
        dw_post = _dense(dw_post, "dw_post", (D,), torch.float32, dev, stream)
    if w_pre is not None:
        dw_pre = _dense(dw_pre, "dw_pre", (D,), torch.float32, dev, stream)
    for name, given, has in (("dy", dy, y), ("dgate", dgate, gate), ("dw_post", dw_post, w_post),
                             ("dw_pre", dw_pre, w_pre)):
        if given is not None and has is None:
            raise ValueError(f"{name} has no input")
    if workspace is None:
        workspace = _new(_workspace_bytes(fields), torch.uint8, dev, stream)
    _need(workspace, "workspace", device=dev)
    _launch(lib.gdr_block_norm_bwd, "gdr_block_norm_bwd", dev, stream, _shape(fields), _addr(dx_out), _addr(dh),
            x_out.data_ptr(), _addr(y), _addr(gate), _addr(w_post), _addr(w_pre), dx.data_ptr(), _addr(dy),
            _addr(dgate), _addr(dw_post), _addr(dw_pre), workspace.data_ptr(), workspace.nbytes)
    return dx, dy, dgate, dw_post, dw_pre
