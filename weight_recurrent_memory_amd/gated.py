"""ctypes binding of the gated linear recurrence (falcon_gated_* of libfalcon):

    S_t = a_t S_{t-1} + v_t k_t^T,   a_t = exp(log_a_t),   o_t = S_t q_t
"""
from __future__ import annotations

from . import binding as _b


def _sizes(torch, q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4 or not q.is_cuda:
        raise ValueError("q, k, v must be [batch, heads, L, d] on a GPU")
    B, H, L, dk = q.shape
    return B, H, L, dk, v.shape[-1], _b._dtype_code(torch, q)


def _inputs(torch, q, k, v, log_a, S0, sizes):
    """Checked addresses of q, k, v, log_a, S0."""
    B, H, L, dk, dv, _ = sizes
    dev, dt, f32 = q.device, q.dtype, torch.float32
    return (_b._expect(torch, "q", q, (B, H, L, dk), dt, dev),
            _b._expect(torch, "k", k, (B, H, L, dk), dt, dev),
            _b._expect(torch, "v", v, (B, H, L, dv), dt, dev),
            _b._expect(torch, "log_a", log_a, (B, H, L), f32, dev),
            _b._expect(torch, "S0", S0, (B, H, dv, dk), f32, dev))


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
    return workspace, _b._address(workspace), workspace.numel() * workspace.element_size()


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
    sizes = B, H, L, dk, dv, dcode = _sizes(torch, q, k, v)
    dev, f32 = q.device, torch.float32
    ins = _inputs(torch, q, k, v, log_a, S0, sizes)
    with _b._guard(torch, dev, stream):
        if out is None:
            out = q.new_empty((B, H, L, dv), dtype=f32)
            op = out.data_ptr()
        else:
            op = _b._expect(torch, "out", out, (B, H, L, dv), f32, dev)
        if S_out is None and return_state:
            S_out = q.new_empty((B, H, dv, dk), dtype=f32)
        Sp = _b._expect(torch, "S_out", S_out, (B, H, dv, dk), f32, dev)
        need = 0
        if workspace is not None:
            need = lib.falcon_gated_fwd_workspace_bytes(*sizes)
        ws, wp, wb = _workspace(torch, workspace, need, dev)
        status = lib.falcon_gated_fwd_chunk(*sizes, *ins, op, Sp, wp, wb,
                                            _b._raw_stream(torch, dev, stream))
    _b._raise(lib, "falcon_gated_fwd_chunk", status)
    return (out, S_out) if return_state else out


def gated_bwd_chunk(q, k, v, log_a, dO, *, S0=None, dS_L=None, stream=None, workspace="auto"):
    """Gradients of sum <dO, o> + <dS_L, S_L>: a dict of float32 tensors dq, dk, dv, and
    dlog_a / dS0 when log_a / S0 are given.  dO [B,H,L,dv] and dS_L [B,H,dv,dk] float32.
    workspace: "auto", or a device tensor of falcon_gated_bwd_workspace_bytes(...)."""
    import torch
    lib = _b.load_library()
    sizes = B, H, L, dk, dv, dcode = _sizes(torch, q, k, v)
    dev, f32 = q.device, torch.float32
    ins = _inputs(torch, q, k, v, log_a, S0, sizes)
    if dO is None:
        raise ValueError("dO must be given")
    dOp = _b._expect(torch, "dO", dO, (B, H, L, dv), f32, dev)
    dSp = _b._expect(torch, "dS_L", dS_L, (B, H, dv, dk), f32, dev)
    with _b._guard(torch, dev, stream):
        res = dict(dq=q.new_empty((B, H, L, dk), dtype=f32), dk=q.new_empty((B, H, L, dk), dtype=f32),
                   dv=q.new_empty((B, H, L, dv), dtype=f32))
        if log_a is not None:
            res["dlog_a"] = q.new_empty((B, H, L), dtype=f32)
        if S0 is not None:
            res["dS0"] = q.new_empty((B, H, dv, dk), dtype=f32)
        need = lib.falcon_gated_bwd_workspace_bytes(*sizes)
        ws, wp, wb = _workspace(torch, workspace, max(need, 16), dev)
        status = lib.falcon_gated_bwd_chunk(
            *sizes, *ins, dOp, dSp, res["dq"].data_ptr(), res["dk"].data_ptr(),
            res["dv"].data_ptr(), _b._address(res.get("dlog_a")), _b._address(res.get("dS0")), wp,
            wb, _b._raw_stream(torch, dev, stream))
    _b._raise(lib, "falcon_gated_bwd_chunk", status)
    return res


def gated_decode_step(S, q, k, v, log_a=None, *, out=None, stream=None):
    """One token: S [N,H,dv,dk] float32 is updated in place, returns o [N,H,dv] float32.
    q, k [N,H,dk], v [N,H,dv] bfloat16 or float32; log_a [N,H] float32, None: no decay."""
    import torch
    lib = _b.load_library()
    if S.dim() != 4 or not S.is_cuda:
        raise ValueError("S must be [nseq, heads, dv, dk] on a GPU")
    N, H, dv, dk = S.shape
    dev, dt, f32 = S.device, q.dtype, torch.float32
    dcode = _b._dtype_code(torch, q)
    ins = (_b._expect(torch, "S", S, (N, H, dv, dk), f32, dev),
           _b._expect(torch, "q", q, (N, H, dk), dt, dev),
           _b._expect(torch, "k", k, (N, H, dk), dt, dev),
           _b._expect(torch, "v", v, (N, H, dv), dt, dev),
           _b._expect(torch, "log_a", log_a, (N, H), f32, dev))
    with _b._guard(torch, dev, stream):
        if out is None:
            out = S.new_empty((N, H, dv))
            op = out.data_ptr()
        else:
            op = _b._expect(torch, "out", out, (N, H, dv), f32, dev)
        status = lib.falcon_gated_decode_step(N, H, dk, dv, dcode, *ins, op,
                                              _b._raw_stream(torch, dev, stream))
    _b._raise(lib, "falcon_gated_decode_step", status)
    return out
