"""ctypes binding of the gated linear recurrence (falcon_gated_* of libfalcon):

    S_t = a_t S_{t-1} + v_t k_t^T,   a_t = exp(log_a_t),   o_t = S_t q_t
"""
from __future__ import annotations

from . import binding as _b


def gated_decode_step(S, q, k, v, log_a=None, *, out=None, stream=None):
    """One token: S [N,H,dv,dk] float32 is updated in place, returns o [N,H,dv] float32.
    q, k [N,H,dk], v [N,H,dv] bfloat16 or float32; log_a [N,H] float32, None: no decay."""
    import torch
    lib = _b.load_library()
    if S.dim() != 4:
        raise ValueError("S must be [nseq, heads, dv, dk]")
    N, H, dv, dk = S.shape
    dev, dt, f32 = S.device, q.dtype, torch.float32
    dcode = _b._dtype_code(torch, q)
    _b._check(torch, "S", S, (N, H, dv, dk), f32, dev)
    _b._check(torch, "q", q, (N, H, dk), dt, dev)
    _b._check(torch, "k", k, (N, H, dk), dt, dev)
    _b._check(torch, "v", v, (N, H, dv), dt, dev)
    _b._check(torch, "log_a", log_a, (N, H), f32, dev)
    with _b._guard(torch, dev, stream):
        if out is None:
            out = torch.empty((N, H, dv), device=dev, dtype=f32)
        else:
            _b._check(torch, "out", out, (N, H, dv), f32, dev)
        status = lib.falcon_gated_decode_step(N, H, dk, dv, dcode, _b._ptr(S), _b._ptr(q),
                                              _b._ptr(k), _b._ptr(v), _b._ptr(log_a), _b._ptr(out),
                                              _b._stream(torch, dev, stream))
    _b._raise(lib, "falcon_gated_decode_step", status)
    return out
