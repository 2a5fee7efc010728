"""Plain fp64 numpy forms of the gated delta rule and of rotary positions (test
infrastructure; shares no code with the HIP path).

Gated delta rule, per (batch, head), one token at a time:
    S_t = a_t S_{t-1} + u_t k_t^T,   u_t = beta_t (v_t - a_t S_{t-1} k_t),   o_t = S_t q_t
Rotary positions, per token, head and pair of columns:
    (x1, x2) -> scale (x1 cos - x2 sin, x2 cos + x1 sin),   angle = position * frequency
"""
import numpy as np

from oracle.block_oracle import _decay, _f64, unit_rows, unit_rows_backward


def delta_recurrence(q, k, v, beta, log_a=None, S0=None):
    """o [B,H,L,dv] and S_L [B,H,dv,dk]."""
    q, k, v, b = _f64(q), _f64(k), _f64(v), _f64(beta)
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    a = _decay(log_a, (B, H, L))
    S = np.zeros((B, H, dv, dk)) if S0 is None else _f64(S0).copy()
    o = np.empty((B, H, L, dv))
    for t in range(L):
        S = a[:, :, t, None, None] * S
        u = b[:, :, t, None] * (v[:, :, t] - np.einsum("bhij,bhj->bhi", S, k[:, :, t]))
        S = S + u[..., :, None] * k[:, :, t, None, :]
        o[:, :, t] = np.einsum("bhij,bhj->bhi", S, q[:, :, t])
    return o, S


def delta_backward(q, k, v, beta, log_a, dO, S0=None, dS_L=None):
    """Gradients of sum <dO, o> + <dS_L, S_L>, in reverse with the stored states."""
    q, k, v, b, dO = _f64(q), _f64(k), _f64(v), _f64(beta), _f64(dO)
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    a = _decay(log_a, (B, H, L))
    states, errs = [np.zeros((B, H, dv, dk)) if S0 is None else _f64(S0)], []
    for t in range(L):
        S = a[:, :, t, None, None] * states[-1]
        errs.append(v[:, :, t] - np.einsum("bhij,bhj->bhi", S, k[:, :, t]))
        states.append(S + (b[:, :, t, None] * errs[-1])[..., :, None] * k[:, :, t, None, :])
    R = np.zeros((B, H, dv, dk)) if dS_L is None else _f64(dS_L).copy()
    out = dict(dq=np.empty_like(q), dk=np.empty_like(k), dv=np.empty_like(v),
               dbeta=np.empty((B, H, L)), dlog_a=np.empty((B, H, L)))
    for t in range(L - 1, -1, -1):
        bt = b[:, :, t, None]
        R = R + dO[:, :, t, :, None] * q[:, :, t, None, :]
        before = a[:, :, t, None, None] * states[t]
        du = np.einsum("bhij,bhj->bhi", R, k[:, :, t])
        out["dq"][:, :, t] = np.einsum("bhij,bhi->bhj", states[t + 1], dO[:, :, t])
        out["dk"][:, :, t] = bt * (np.einsum("bhij,bhi->bhj", R, errs[t])
                                   - np.einsum("bhij,bhi->bhj", before, du))
        out["dv"][:, :, t] = bt * du
        out["dbeta"][:, :, t] = np.sum(du * errs[t], -1)
        R = R - (bt * du)[..., :, None] * k[:, :, t, None, :]
        out["dlog_a"][:, :, t] = np.sum(R * before, axis=(2, 3))
        R = a[:, :, t, None, None] * R
    out["dS0"] = R
    return out


def turn(x, positions, freqs, pairs="half", scale=1.0):
    """x [B,H,L,d], its first 2 len(freqs) columns turned by positions [B,L] * freqs."""
    y = _f64(x).copy()
    n = len(freqs)
    i, j = (slice(0, n), slice(n, 2 * n)) if pairs == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    angle = np.asarray(positions, dtype=np.float64)[:, None, :, None] * _f64(freqs)
    c, s = scale * np.cos(angle), scale * np.sin(angle)
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


def rotary_in(x, positions, freqs, pairs="half", scale=1.0, normalize=True, eps=1e-6):
    """x [B,L,H,d] to unit rows, turned, [B,H,L,d]."""
    y = np.swapaxes(unit_rows(x, eps) if normalize else _f64(x), 1, 2)
    return turn(y, positions, freqs, pairs, scale)


def rotary_in_backward(x, dy, positions, freqs, pairs="half", scale=1.0, normalize=True, eps=1e-6):
    """dy [B,H,L,d] to the gradient of x [B,L,H,d]."""
    dx = np.swapaxes(turn(dy, -np.asarray(positions), freqs, pairs, scale), 1, 2)
    return unit_rows_backward(x, dx, eps) if normalize else dx
