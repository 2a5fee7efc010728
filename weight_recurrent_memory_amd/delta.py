"""ctypes binding of the gated delta rule (falcon_gated_delta_* of libfalcon_block):

    S_t = a_t S_{t-1} + u_t k_t^T,   u_t = beta_t (v_t - a_t S_{t-1} k_t),
    o_t = S_t q_t,                   a_t = exp(log_a_t)
"""
from __future__ import annotations

from . import binding as _b
from . import block_binding as _bb
from .gated import _inputs, _sizes, _workspace


def gated_delta_fwd_chunk(q, k, v, beta, log_a=None, *, S0=None, out=None, S_out=None,
                          return_state=False, stream=None, workspace="auto"):
    """o [B,H,L,dv] float32, then S_L [B,H,dv,dk] with return_state.  q, k [B,H,L,dk],
    v [B,H,L,dv] bfloat16 or float32; beta [B,H,L] float32, the write strength; log_a
    [B,H,L] float32 (-inf resets the state), None: no decay; S0: the state to go on from.
    S_out may be S0 (in place).  workspace: "auto" (default) allocates it, or a device
    tensor of falcon_gated_delta_fwd_workspace_bytes(...)."""
    import torch
    lib = _bb.load_library()
    sizes = B, H, L, dk, dv, dcode = _sizes(torch, q, k, v)
    dev, f32 = q.device, torch.float32
    qp, kp, vp, lp, sp = _inputs(torch, q, k, v, log_a, S0, sizes)
    if beta is None:
        raise ValueError("beta must be given")
    bp = _b._expect(torch, "beta", beta, (B, H, L), f32, dev)
    with _b._guard(torch, dev, stream):
        if out is None:
            out = q.new_empty((B, H, L, dv), dtype=f32)
            op = out.data_ptr()
        else:
            op = _b._expect(torch, "out", out, (B, H, L, dv), f32, dev)
        if S_out is None and return_state:
            S_out = q.new_empty((B, H, dv, dk), dtype=f32)
        Sp = _b._expect(torch, "S_out", S_out, (B, H, dv, dk), f32, dev)
        need = lib.falcon_gated_delta_fwd_workspace_bytes(*sizes)
        ws, wp, wb = _workspace(torch, workspace, max(need, 16), dev)
        status = lib.falcon_gated_delta_fwd_chunk(*sizes, qp, kp, vp, bp, lp, sp, op, Sp, wp, wb,
                                                  _b._raw_stream(torch, dev, stream))
    _bb.check("falcon_gated_delta_fwd_chunk", status)
    return (out, S_out) if return_state else out


def gated_delta_bwd_chunk(q, k, v, beta, log_a, dO, *, S0=None, dS_L=None, stream=None,
                          workspace="auto"):
    """Gradients of sum <dO, o> + <dS_L, S_L>: a dict of float32 tensors dq, dk, dv, dbeta,
    and dlog_a / dS0 when log_a / S0 are given.  dO [B,H,L,dv] and dS_L [B,H,dv,dk] float32.
    workspace: "auto", or a device tensor of falcon_gated_delta_bwd_workspace_bytes(...)."""
    import torch
    lib = _bb.load_library()
    sizes = B, H, L, dk, dv, dcode = _sizes(torch, q, k, v)
    dev, f32 = q.device, torch.float32
    qp, kp, vp, lp, sp = _inputs(torch, q, k, v, log_a, S0, sizes)
    if beta is None or dO is None:
        raise ValueError("beta and dO must be given")
    bp = _b._expect(torch, "beta", beta, (B, H, L), f32, dev)
    dOp = _b._expect(torch, "dO", dO, (B, H, L, dv), f32, dev)
    dSp = _b._expect(torch, "dS_L", dS_L, (B, H, dv, dk), f32, dev)
    with _b._guard(torch, dev, stream):
        res = dict(dq=q.new_empty((B, H, L, dk), dtype=f32), dk=q.new_empty((B, H, L, dk), dtype=f32),
                   dv=q.new_empty((B, H, L, dv), dtype=f32), dbeta=q.new_empty((B, H, L), dtype=f32))
        if log_a is not None:
            res["dlog_a"] = q.new_empty((B, H, L), dtype=f32)
        if S0 is not None:
            res["dS0"] = q.new_empty((B, H, dv, dk), dtype=f32)
        need = lib.falcon_gated_delta_bwd_workspace_bytes(*sizes)
        ws, wp, wb = _workspace(torch, workspace, max(need, 16), dev)
        status = lib.falcon_gated_delta_bwd_chunk(
            *sizes, qp, kp, vp, bp, lp, sp, dOp, dSp, res["dq"].data_ptr(), res["dk"].data_ptr(),
            res["dv"].data_ptr(), res["dbeta"].data_ptr(), _b._address(res.get("dlog_a")),
            _b._address(res.get("dS0")), wp, wb, _b._raw_stream(torch, dev, stream))
    _bb.check("falcon_gated_delta_bwd_chunk", status)
    return res


def gated_delta_decode_step(S, q, k, v, beta, log_a=None, *, out=None, stream=None):
    """One token: S [N,H,dv,dk] float32 is updated in place, returns o [N,H,dv] float32.
    q, k [N,H,dk], v [N,H,dv] bfloat16 or float32; beta and log_a [N,H] float32, log_a
    None: no decay."""
    import torch
    lib = _bb.load_library()
    if S.dim() != 4 or not S.is_cuda:
        raise ValueError("S must be [nseq, heads, dv, dk] on a GPU")
    if beta is None:
        raise ValueError("beta must be given")
    N, H, dv, dk = S.shape
    dev, dt, f32 = S.device, q.dtype, torch.float32
    dcode = _b._dtype_code(torch, q)
    ins = (_b._expect(torch, "S", S, (N, H, dv, dk), f32, dev),
           _b._expect(torch, "q", q, (N, H, dk), dt, dev),
           _b._expect(torch, "k", k, (N, H, dk), dt, dev),
           _b._expect(torch, "v", v, (N, H, dv), dt, dev),
           _b._expect(torch, "beta", beta, (N, H), f32, dev),
           _b._expect(torch, "log_a", log_a, (N, H), f32, dev))
    with _b._guard(torch, dev, stream):
        if out is None:
            out = S.new_empty((N, H, dv))
            op = out.data_ptr()
        else:
            op = _b._expect(torch, "out", out, (N, H, dv), f32, dev)
        status = lib.falcon_gated_delta_decode_step(N, H, dk, dv, dcode, *ins, op,
                                                    _b._raw_stream(torch, dev, stream))
    _bb.check("falcon_gated_delta_decode_step", status)
    return out
