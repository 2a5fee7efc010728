"""ctypes binding of rotary positions at a block's entry (falcon_rotary_in of
libfalcon_block), and the frequencies that it takes.

norm_in with the first columns of every q and k row turned, in pairs, by an angle
proportional to the token's position.  Layouts as norms.py's.
"""
from __future__ import annotations

import math

from . import binding as _b
from . import block_binding as _bb
from .norms import _rows, _token_major

PAIRS = {"half": 0, "neighbours": 1}


def rotary_frequencies(rot, base=10000.0, *, scaling=None, factor=1.0, original_length=None,
                       slow=1.0, fast=32.0, device=None):
    """The rot / 2 frequencies, radians a token, float64: base^(-2 i / rot).  scaling, for
    sequences `factor` times as long as those a model was trained on:
      "linear"   every frequency divided by factor
      "base"     base grown by factor^(rot / (rot - 2)): the first pair keeps its frequency,
                 the last one's is divided by factor
      "by_turns" pairs that turn at most `slow` times over original_length tokens divided by
                 factor, those that turn `fast` times or more left, between them in between"""
    import torch
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2, got %r" % (rot,))
    if not (base > 0 and math.isfinite(base)) or not (factor > 0 and math.isfinite(factor)):
        raise ValueError("base and factor must be positive")
    if scaling == "base":
        if rot < 4:
            raise ValueError("scaling by the base needs two pairs at least")
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_turns":
        if not original_length or original_length <= 0 or not fast > slow:
            raise ValueError("scaling by turns needs original_length, and fast above slow")
        left = ((original_length * f / (2.0 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * left + f / factor * (1.0 - left)
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'by_turns', got %r" % (scaling,))
    return f.to(device)


def _rotation(torch, positions, freqs, pairs, normalize, B, L, dev):
    """(positions, freqs, rot, pairs, normalize) as the library takes them."""
    if pairs not in PAIRS:
        raise ValueError("pairs must be one of %s, got %r" % (sorted(PAIRS), pairs))
    if positions is None or freqs is None:
        raise ValueError("positions and freqs must be given")
    if freqs.dim() != 1:
        raise ValueError("freqs must be [rot / 2]")
    pp = _b._expect(torch, "positions", positions, (B, L), torch.int64, dev)
    fp = _b._expect(torch, "freqs", freqs, (freqs.shape[0],), torch.float64, dev)
    return pp, fp, 2 * freqs.shape[0], PAIRS[pairs], 1 if normalize else 0


def rotary_in(q_in, k_in, v_in, positions, freqs, *, pairs="half", scale=1.0, normalize=True,
              eps=1e-6, out=None, stream=None):
    """(q, k, v) head-major [B,H,L,d] from token-major q_in, k_in, v_in [B,L,H,d] (bfloat16
    or float32; v_in or None): q = q_in / sqrt(|q_in|^2 + eps) (normalize=False: q_in), its
    first 2 * len(freqs) columns turned by positions * freqs and times scale; k likewise,
    v = v_in.  positions [B,L] int64, freqs [rot / 2] float64 (rotary_frequencies).  pairs:
    "half" (columns i and i + rot / 2) or "neighbours" (2 i and 2 i + 1).  out: the three
    results."""
    import torch
    lib = _bb.load_library()
    _token_major(torch, "q_in", q_in)
    B, L, H, dk = q_in.shape
    dev, dt = q_in.device, q_in.dtype
    dcode = _b._dtype_code(torch, q_in)
    dv = dk if v_in is None else v_in.shape[-1]
    qp, ldq = _rows(torch, "q_in", q_in, (B, L, H, dk), dt, dev)
    kp, ldk = _rows(torch, "k_in", k_in, (B, L, H, dk), dt, dev)
    vp, ldv = _rows(torch, "v_in", v_in, (B, L, H, dv), dt, dev)
    pp, fp, rot, kind, norm = _rotation(torch, positions, freqs, pairs, normalize, B, L, dev)
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
        status = lib.falcon_rotary_in(B, H, L, dk, dv, dcode, qp, ldq, kp, ldk, vp, ldv, pp, fp, rot,
                                      kind, float(scale), norm, float(eps), _b._address(q),
                                      _b._address(k), _b._address(v), _b._raw_stream(torch, dev, stream))
    _bb.check("falcon_rotary_in", status)
    return q, k, v


def rotary_in_bwd(q_in, k_in, dq, dk, dv, positions, freqs, *, pairs="half", scale=1.0,
                  normalize=True, eps=1e-6, out=None, stream=None):
    """Gradients of rotary_in: dq, dk, dv [B,H,L,d] float32 (dv or None) to (dq_in, dk_in,
    dv_in) [B,L,H,d] in q_in's type.  out: the three results, which may be views of one
    fused buffer."""
    import torch
    lib = _bb.load_library()
    _token_major(torch, "q_in", q_in)
    B, L, H, ndk = q_in.shape
    dev, dt, f32 = q_in.device, q_in.dtype, torch.float32
    dcode = _b._dtype_code(torch, q_in)
    ndv = ndk if dv is None else dv.shape[-1]
    qp, ldq = _rows(torch, "q_in", q_in, (B, L, H, ndk), dt, dev)
    kp, ldk = _rows(torch, "k_in", k_in, (B, L, H, ndk), dt, dev)
    if dq is None or dk is None:
        raise ValueError("dq and dk must be given")
    dqp = _b._expect(torch, "dq", dq, (B, H, L, ndk), f32, dev)
    dkp = _b._expect(torch, "dk", dk, (B, H, L, ndk), f32, dev)
    dvp = _b._expect(torch, "dv", dv, (B, H, L, ndv), f32, dev)
    pp, fp, rot, kind, norm = _rotation(torch, positions, freqs, pairs, normalize, B, L, dev)
    with _b._guard(torch, dev, stream):
        if out is None:
            out = (q_in.new_empty((B, L, H, ndk)), q_in.new_empty((B, L, H, ndk)),
                   None if dv is None else q_in.new_empty((B, L, H, ndv)))
        oqp, ldoq = _rows(torch, "out[0]", out[0], (B, L, H, ndk), dt, dev)
        okp, ldok = _rows(torch, "out[1]", out[1], (B, L, H, ndk), dt, dev)
        ovp, ldov = _rows(torch, "out[2]", out[2], (B, L, H, ndv), dt, dev)
        status = lib.falcon_rotary_in_bwd(B, H, L, ndk, ndv, dcode, qp, ldq, kp, ldk, pp, fp, rot, kind,
                                          float(scale), norm, float(eps), dqp, dkp, dvp, oqp, ldoq, okp,
                                          ldok, ovp, ldov, _b._raw_stream(torch, dev, stream))
    _bb.check("falcon_rotary_in_bwd", status)
    return tuple(out)
