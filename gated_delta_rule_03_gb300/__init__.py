"""GB300-native gated delta rule (Gated DeltaNet recurrence).

The compute path is the C-ABI library `libgdr.so` (hand-written sm_103a CUDA,
declared in include/gdr.h). This package is a thin binding over it:

    from gated_delta_rule_03_gb300 import chunk_fwd, decode_step
    from gated_delta_rule_03_gb300 import linattn_fwd, linattn_bwd, linattn_step
    from gated_delta_rule_03_gb300 import block_norm_fwd, block_norm_bwd

Importing the package loads nothing; the first call loads the library and
raises if it is missing. There is no CPU fallback. The submodule `inputs`
(seeded synthetic inputs) can be imported on its own.
"""
_OPS = ("GdrError", "chunk_fwd", "chunk_fwd_workspace_size", "decode_step", "library_path",
        "read_device_status", "status_string")
_LINATTN = ("linattn_fwd", "linattn_fwd_workspace_size", "linattn_bwd", "linattn_bwd_workspace_size",
            "linattn_step")
_BLOCK_NORM = ("block_norm_fwd", "block_norm_bwd", "block_norm_bwd_workspace_size")

__all__ = list(_OPS + _LINATTN + _BLOCK_NORM)


def __getattr__(name):
    for names, module in ((_OPS, "ops"), (_LINATTN, "linattn"), (_BLOCK_NORM, "block_norm")):
        if name in names:
            from importlib import import_module
            globals()[name] = found = getattr(import_module("." + module, __name__), name)
            return found  # (kept: the next look-up does not come here, 3 us of a small call)
    raise AttributeError(name)
