"""ctypes binding of the gated linear recurrence (falcon_gated_* of libfalcon):

    S_t = a_t S_{t-1} + v_t k_t^T,   a_t = exp(log_a_t),   o_t = S_t q_t
"""
from __future__ import annotations

from . import binding as _b


def _inputs(torch, q, k, v, log_a, S0):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [batch, heads, L, d]")
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    dev, dt, f32 = q.device, q.dtype, torch.float32
    dcode = _b._dtype_code(torch, q)
    _b._check(torch, "q", q, (B, H, L, dk), dt, dev)
    _b._check(torch, "k", k, (B, H, L, dk), dt, dev)
    _b._check(torch, "v", v, (B, H, L, dv), dt, dev)
    _b._check(torch, "log_a", log_a, (B, H, L), f32, dev)
    _b._check(torch, "S0", S0, (B, H, dv, dk), f32, dev)
    return B, H, L, dk, dv, dcode


def _workspace(torch, workspace, need, dev):
    """(tensor kept alive, pointer, bytes) of a workspace argument."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace: None, 'auto' or a device tensor")
        workspace = torch.empty(need, device=dev, dtype=torch.uint8) if need > 0 else None
    if workspace is None:
        return None, None, 0
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace, _b._ptr(workspace), workspace.numel() * workspace.element_size()


def gated_fwd_chunk(q, k, v, log_a=None, *, S0=None, out=None, S_out=None, return_state=False,
                    stream=None, workspace="auto"):
    """o [B,H,L,dv] float32, then S_L [B,H,dv,dk] with return_state.  q, k [B,H,L,dk],
    v [B,H,L,dv] bfloat16 or float32; log_a [B,H,L] float32 (-inf resets the state),
    None: no decay; S0: the state to go on from.  S_out may be S0 (in place).
    workspace: "auto" (default) allocates what cuts a long sequence of few heads into
    segments (falcon_gated_fwd_workspace_bytes), a device tensor supplies it, None
    walks each sequence in order."""
    import torch
    lib = _b.load_library()
    B, H, L, dk, dv, dcode = _inputs(torch, q, k, v, log_a, S0)
    dev, f32 = q.device, torch.float32
    with _b._guard(torch, dev, stream):
        if out is None:
            out = torch.empty((B, H, L, dv), device=dev, dtype=f32)
        else:
            _b._check(torch, "out", out, (B, H, L, dv), f32, dev)
        if S_out is None:
            S_out = torch.empty((B, H, dv, dk), device=dev, dtype=f32) if return_state else None
        else:
            _b._check(torch, "S_out", S_out, (B, H, dv, dk), f32, dev)
        need = 0
        if workspace is not None:
            need = lib.falcon_gated_fwd_workspace_bytes(B, H, L, dk, dv, dcode)
        ws, wp, wb = _workspace(torch, workspace, need, dev)
        status = lib.falcon_gated_fwd_chunk(B, H, L, dk, dv, dcode, _b._ptr(q), _b._ptr(k),
                                            _b._ptr(v), _b._ptr(log_a), _b._ptr(S0), _b._ptr(out),
                                            _b._ptr(S_out), wp, wb, _b._stream(torch, dev, stream))
    _b._raise(lib, "falcon_gated_fwd_chunk", status)
    return (out, S_out) if return_state else out


def gated_bwd_chunk(q, k, v, log_a, dO, *, S0=None, dS_L=None, stream=None, workspace="auto"):
    """Gradients of sum <dO, o> + <dS_L, S_L>: a dict of float32 tensors dq, dk, dv, and
    dlog_a / dS0 when log_a / S0 are given.  dO [B,H,L,dv] and dS_L [B,H,dv,dk] float32.
    workspace: "auto", or a device tensor of falcon_gated_bwd_workspace_bytes(...)."""
    import torch
    lib = _b.load_library()
    B, H, L, dk, dv, dcode = _inputs(torch, q, k, v, log_a, S0)
    dev, f32 = q.device, torch.float32
    if dO is None:
        raise ValueError("dO must be given")
    _b._check(torch, "dO", dO, (B, H, L, dv), f32, dev)
    _b._check(torch, "dS_L", dS_L, (B, H, dv, dk), f32, dev)
    with _b._guard(torch, dev, stream):
        res = dict(dq=torch.empty((B, H, L, dk), device=dev, dtype=f32),
                   dk=torch.empty((B, H, L, dk), device=dev, dtype=f32),
                   dv=torch.empty((B, H, L, dv), device=dev, dtype=f32))
        if log_a is not None:
            res["dlog_a"] = torch.empty((B, H, L), device=dev, dtype=f32)
        if S0 is not None:
            res["dS0"] = torch.empty((B, H, dv, dk), device=dev, dtype=f32)
        need = lib.falcon_gated_bwd_workspace_bytes(B, H, L, dk, dv, dcode)
        ws, wp, wb = _workspace(torch, workspace, max(int(need), 16), dev)
        status = lib.falcon_gated_bwd_chunk(
            B, H, L, dk, dv, dcode, _b._ptr(q), _b._ptr(k), _b._ptr(v), _b._ptr(log_a), _b._ptr(S0),
            _b._ptr(dO), _b._ptr(dS_L), _b._ptr(res["dq"]), _b._ptr(res["dk"]), _b._ptr(res["dv"]),
            _b._ptr(res.get("dlog_a")), _b._ptr(res.get("dS0")), wp, wb,
            _b._stream(torch, dev, stream))
    _b._raise(lib, "falcon_gated_bwd_chunk", status)
    return res


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
