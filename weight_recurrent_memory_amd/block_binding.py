"""Loading of libfalcon_block, and the pieces that its bindings share with binding.py."""
from __future__ import annotations

import ctypes
import os

from . import binding as _b

_LIB = None


def library_path() -> str:
    return os.path.join(os.path.dirname(_b.library_path()), "libfalcon_block.so")


def load_library():
    """Load libfalcon_block.so from the package directory (built in-tree)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise ImportError("libfalcon_block.so not built at %s; run __graft_entry__.build()" % path)
    lib = ctypes.CDLL(path)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    ll, ull = ctypes.c_longlong, ctypes.c_ulonglong
    lib.falcon_gated_delta_fwd_workspace_bytes.restype = ull
    lib.falcon_gated_delta_fwd_workspace_bytes.argtypes = [i] * 6
    lib.falcon_gated_delta_fwd_chunk.restype = i
    lib.falcon_gated_delta_fwd_chunk.argtypes = [i] * 6 + [vp] * 9 + [ull, vp]
    lib.falcon_gated_delta_bwd_workspace_bytes.restype = ull
    lib.falcon_gated_delta_bwd_workspace_bytes.argtypes = [i] * 6
    lib.falcon_gated_delta_bwd_chunk.restype = i
    lib.falcon_gated_delta_bwd_chunk.argtypes = [i] * 6 + [vp] * 15 + [ull, vp]
    lib.falcon_gated_delta_decode_step.restype = i
    lib.falcon_gated_delta_decode_step.argtypes = [i] * 5 + [vp] * 8
    lib.falcon_rotary_in.restype = i
    lib.falcon_rotary_in.argtypes = [i] * 6 + [vp, ll, vp, ll, vp, ll, vp, vp, i, i, f, i, f] + [vp] * 4
    lib.falcon_rotary_in_bwd.restype = i
    lib.falcon_rotary_in_bwd.argtypes = [i] * 6 + [vp, ll, vp, ll, vp, vp, i, i, f, i, f, vp, vp, vp,
                                                   vp, ll, vp, ll, vp, ll, vp]
    _LIB = lib
    return lib


def check(fn, status):
    """Raises FalconError for a status other than ok."""
    if status != 0:
        _b._raise(_b.load_library(), fn, status)
