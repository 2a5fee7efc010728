"""ctypes binding of the norms before and after a block (falcon_norm_* of libfalcon).

Token-major tensors [B, L, H, d] may be views of one fused projection: the last
dimension contiguous, heads d apart, tokens any multiple of 16 bytes apart, batch
after batch.  Head-major tensors [B, H, L, d] are contiguous, as the sequence
entry points take them.
"""
from __future__ import annotations

from . import binding as _b

GATE_KINDS = {"silu": 0, "sigmoid": 1}


def _rows(torch, name, t, shape, dtype, device):
    """Checks a token-major tensor; returns (pointer, ld)."""
    if t is None:
        return None, 0
    if t.device != device:
        raise ValueError("%s must live on %s" % (name, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s shape %s != %s" % (name, tuple(t.shape), shape))
    B, L, H, d = shape
    s0, s1, s2, s3 = t.stride()
    ld = H * d if B * L == 1 else (s0 if L == 1 else s1)
    if s3 != 1 or (H > 1 and s2 != d) or ld < H * d or (B > 1 and s0 != L * ld):
        raise ValueError("%s: strides %s of %s are not rows of %d elements at one distance"
                         % (name, t.stride(), shape, H * d))
    at = t.data_ptr()
    if at % 16 or ld * t.element_size() % 16:
        raise ValueError("%s: rows must start 16-byte aligned and lie a multiple of 16 bytes "
                         "apart (%d elements of %s)" % (name, ld, dtype))
    return at, ld


def _token_major(torch, name, t):
    if t.dim() != 4:
        raise ValueError("%s must be [batch, L, heads, d]" % name)
    if not t.is_cuda:
        raise ValueError("%s must live on a GPU" % name)


def _gate_kind(kind):
    if kind not in GATE_KINDS:
        raise ValueError("gate_kind must be one of %s, got %r" % (sorted(GATE_KINDS), kind))
    return GATE_KINDS[kind]


def norm_in(q_in, k_in, v_in=None, *, eps=1e-6, out=None, stream=None):
    """q = q_in / sqrt(|q_in|^2 + eps) per token and head, k likewise, v = v_in:
    token-major [B,L,H,d] (bfloat16 or float32) to head-major [B,H,L,d] of the same
    type.  Returns (q, k, v), v None without v_in.  out: the three results."""
    import torch
    lib = _b.load_library()
    _token_major(torch, "q_in", q_in)
    B, L, H, dk = q_in.shape
    dev, dt = q_in.device, q_in.dtype
    dcode = _b._dtype_code(torch, q_in)
    dv = dk if v_in is None else v_in.shape[-1]
    qp, ldq = _rows(torch, "q_in", q_in, (B, L, H, dk), dt, dev)
    kp, ldk = _rows(torch, "k_in", k_in, (B, L, H, dk), dt, dev)
    vp, ldv = _rows(torch, "v_in", v_in, (B, L, H, dv), dt, dev)
    with _b._guard(torch, dev, stream):
        if out is None:
            q = q_in.new_empty((B, H, L, dk))
            k = q_in.new_empty((B, H, L, dk))
            v = None if v_in is None else q_in.new_empty((B, H, L, dv))
        else:
            q, k, v = out
            if q is None or k is None:
                raise ValueError("out must hold q and k")
            _b._expect(torch, "out[0]", q, (B, H, L, dk), dt, dev)
            _b._expect(torch, "out[1]", k, (B, H, L, dk), dt, dev)
            _b._expect(torch, "out[2]", v, (B, H, L, dv), dt, dev)
        status = lib.falcon_norm_in(B, H, L, dk, dv, dcode, qp, ldq, kp, ldk, vp, ldv, float(eps),
                                    _b._address(q), _b._address(k), _b._address(v),
                                    _b._raw_stream(torch, dev, stream))
    _b._raise(lib, "falcon_norm_in", status)
    return q, k, v


def norm_in_bwd(q_in, k_in, dq, dk, dv=None, *, eps=1e-6, out=None, stream=None):
    """Gradients of norm_in: dq, dk, dv [B,H,L,d] float32 (as bwd_chunk and
    gated_bwd_chunk give them) to (dq_in, dk_in, dv_in) [B,L,H,d] in q_in's type, dv_in
    None without dv.  out: the three results, which may be views of one fused buffer."""
    import torch
    lib = _b.load_library()
    _token_major(torch, "q_in", q_in)
    B, L, H, ndk = q_in.shape
    dev, dt, f32 = q_in.device, q_in.dtype, torch.float32
    dcode = _b._dtype_code(torch, q_in)
    ndv = ndk if dv is None else dv.shape[-1]
    qp, ldq = _rows(torch, "q_in", q_in, (B, L, H, ndk), dt, dev)
    kp, ldk = _rows(torch, "k_in", k_in, (B, L, H, ndk), dt, dev)
    if dq is None or dk is None:
        raise ValueError("dq and dk must be given")
    _b._expect(torch, "dq", dq, (B, H, L, ndk), f32, dev)
    _b._expect(torch, "dk", dk, (B, H, L, ndk), f32, dev)
    _b._expect(torch, "dv", dv, (B, H, L, ndv), f32, dev)
    with _b._guard(torch, dev, stream):
        if out is None:
            out = (q_in.new_empty((B, L, H, ndk)),
                   q_in.new_empty((B, L, H, ndk)),
                   None if dv is None else q_in.new_empty((B, L, H, ndv)))
        oqp, ldoq = _rows(torch, "out[0]", out[0], (B, L, H, ndk), dt, dev)
        okp, ldok = _rows(torch, "out[1]", out[1], (B, L, H, ndk), dt, dev)
        ovp, ldov = _rows(torch, "out[2]", out[2], (B, L, H, ndv), dt, dev)
        status = lib.falcon_norm_in_bwd(B, H, L, ndk, ndv, dcode, qp, ldq, kp, ldk, float(eps),
                                        _b._address(dq), _b._address(dk), _b._address(dv), oqp, ldoq, okp,
                                        ldok, ovp, ldov, _b._raw_stream(torch, dev, stream))
    _b._raise(lib, "falcon_norm_in_bwd", status)
    return tuple(out)


def norm_out(o, weight, gate=None, *, gate_kind="silu", residual=None, scale=1.0, eps=1e-6,
             dtype=None, out=None, stream=None):
    """y = residual + scale * act(gate) * weight * o / sqrt(mean(o^2) + eps) per token
    and head: o [B,H,L,dv] float32, weight [dv] float32, gate and residual token-major
    [B,L,H,dv] or None (no factor, no addend).  Returns y [B,L,H,dv] in the type of
    out, gate or residual, else dtype (default bfloat16).  out may be residual."""
    import torch
    lib = _b.load_library()
    if o.dim() != 4 or not o.is_cuda:
        raise ValueError("o must be [batch, heads, L, dv] on a GPU")
    B, H, L, dv = o.shape
    dev = o.device
    kind = _gate_kind(gate_kind)
    given = [t.dtype for t in (out, gate, residual) if t is not None]
    dt = given[0] if given else (dtype or torch.bfloat16)
    if dtype is not None and dtype != dt:
        raise TypeError("dtype %s, but the tensors given are %s" % (dtype, dt))
    _b._expect(torch, "o", o, (B, H, L, dv), torch.float32, dev)
    _b._expect(torch, "weight", weight, (dv,), torch.float32, dev)
    gp, ldg = _rows(torch, "gate", gate, (B, L, H, dv), dt, dev)
    rp, ldr = _rows(torch, "residual", residual, (B, L, H, dv), dt, dev)
    with _b._guard(torch, dev, stream):
        if out is None:
            out = o.new_empty((B, L, H, dv), dtype=dt)
        dcode = _b._dtype_code(torch, out)
        yp, ldy = _rows(torch, "out", out, (B, L, H, dv), dt, dev)
        status = lib.falcon_norm_out(B, H, L, dv, dcode, _b._address(o), _b._address(weight), gp, ldg, kind,
                                     rp, ldr, float(scale), float(eps), yp, ldy,
                                     _b._raw_stream(torch, dev, stream))
    _b._raise(lib, "falcon_norm_out", status)
    return out


def norm_out_bwd(o, weight, dy, gate=None, *, gate_kind="silu", scale=1.0, eps=1e-6, dgate=None,
                 stream=None):
    """Gradients of norm_out for dy [B,L,H,dv]: a dict of dO [B,H,L,dv] float32, dweight
    [dv] float32 and, with a gate, dgate [B,L,H,dv] in the gate's type (dgate: a tensor
    to write it to, which may be a view).  The residual's gradient is dy itself."""
    import torch
    lib = _b.load_library()
    if o.dim() != 4 or not o.is_cuda:
        raise ValueError("o must be [batch, heads, L, dv] on a GPU")
    B, H, L, dv = o.shape
    dev, dt, f32 = o.device, dy.dtype, torch.float32
    kind = _gate_kind(gate_kind)
    dcode = _b._dtype_code(torch, dy)
    _b._expect(torch, "o", o, (B, H, L, dv), f32, dev)
    _b._expect(torch, "weight", weight, (dv,), f32, dev)
    dp, ldd = _rows(torch, "dy", dy, (B, L, H, dv), dt, dev)
    gp, ldg = _rows(torch, "gate", gate, (B, L, H, dv), dt, dev)
    if gate is None and dgate is not None:
        raise ValueError("dgate without a gate")
    with _b._guard(torch, dev, stream):
        res = dict(dO=o.new_empty((B, H, L, dv)),
                   dweight=o.new_empty((dv,)))
        if gate is not None:
            res["dgate"] = dgate if dgate is not None else dy.new_empty((B, L, H, dv))
        gop, ldgo = _rows(torch, "dgate", res.get("dgate"), (B, L, H, dv), dt, dev)
        need = int(lib.falcon_norm_out_bwd_workspace_bytes(B, L, dv))
        ws = o.new_empty((max(need, 16) // 4,))
        status = lib.falcon_norm_out_bwd(B, H, L, dv, dcode, _b._address(o), _b._address(weight), gp, ldg,
                                         kind, float(scale), float(eps), dp, ldd,
                                         _b._address(res["dO"]), gop, ldgo, _b._address(res["dweight"]),
                                         _b._address(ws), need, _b._raw_stream(torch, dev, stream))
    _b._raise(lib, "falcon_norm_out_bwd", status)
    return res
