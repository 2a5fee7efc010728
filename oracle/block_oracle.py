"""Plain fp64 numpy forms of the gated linear recurrence and of the norms before and
after a block (test infrastructure; shares no code with the HIP path).

Gated recurrence, per (batch, head), one token at a time:
    S_t = a_t S_{t-1} + v_t k_t^T,   a_t = exp(log_a_t),   o_t = S_t q_t
Norms, per token and head:
    norm_in   y = x / sqrt(|x|^2 + eps)
    norm_out  y = residual + scale act(gate) weight o / sqrt(mean(o^2) + eps)
"""
import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _decay(log_a, shape):
    return np.ones(shape) if log_a is None else np.exp(_f64(log_a))


def gated_recurrence(q, k, v, log_a=None, S0=None):
    """o [B,H,L,dv] and S_L [B,H,dv,dk]."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    a = _decay(log_a, (B, H, L))
    S = np.zeros((B, H, dv, dk)) if S0 is None else _f64(S0).copy()
    o = np.empty((B, H, L, dv))
    for t in range(L):
        S = a[:, :, t, None, None] * S + v[:, :, t, :, None] * k[:, :, t, None, :]
        o[:, :, t] = np.einsum("bhij,bhj->bhi", S, q[:, :, t])
    return o, S


def gated_backward(q, k, v, log_a, dO, S0=None, dS_L=None):
    """Gradients of sum <dO, o> + <dS_L, S_L>, in reverse with the stored states."""
    q, k, v, dO = _f64(q), _f64(k), _f64(v), _f64(dO)
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    a = _decay(log_a, (B, H, L))
    states = [np.zeros((B, H, dv, dk)) if S0 is None else _f64(S0)]
    for t in range(L):
        states.append(a[:, :, t, None, None] * states[-1]
                      + v[:, :, t, :, None] * k[:, :, t, None, :])
    G = np.zeros((B, H, dv, dk)) if dS_L is None else _f64(dS_L).copy()
    out = dict(dq=np.empty_like(q), dk=np.empty_like(k), dv=np.empty_like(v),
               dlog_a=np.empty((B, H, L)))
    for t in range(L - 1, -1, -1):
        G = G + dO[:, :, t, :, None] * q[:, :, t, None, :]
        out["dq"][:, :, t] = np.einsum("bhij,bhi->bhj", states[t + 1], dO[:, :, t])
        out["dk"][:, :, t] = np.einsum("bhij,bhi->bhj", G, v[:, :, t])
        out["dv"][:, :, t] = np.einsum("bhij,bhj->bhi", G, k[:, :, t])
        G = a[:, :, t, None, None] * G
        out["dlog_a"][:, :, t] = np.sum(G * states[t], axis=(2, 3))
    out["dS0"] = G
    return out


def unit_rows(x, eps):
    x = _f64(x)
    return x / np.sqrt(np.sum(x * x, -1, keepdims=True) + eps)


def unit_rows_backward(x, dy, eps):
    x, dy = _f64(x), _f64(dy)
    r = 1.0 / np.sqrt(np.sum(x * x, -1, keepdims=True) + eps)
    y = r * x
    return r * (dy - y * np.sum(y * dy, -1, keepdims=True))


def activation(kind, g):
    """act(g) and act'(g)."""
    g = _f64(g)
    e = np.exp(-np.abs(g))
    s = np.where(g >= 0, 1.0, e) / (1.0 + e)
    if kind == "sigmoid":
        return s, s * (1.0 - s)
    return g * s, s * (1.0 + g * (1.0 - s))


def norm_out(o, weight, gate=None, kind="silu", residual=None, scale=1.0, eps=1e-6):
    """y [B,L,H,dv] from o [B,H,L,dv] and token-major gate and residual."""
    o = np.swapaxes(_f64(o), 1, 2)
    y = scale * _f64(weight) * o / np.sqrt(np.mean(o * o, -1, keepdims=True) + eps)
    if gate is not None:
        y = y * activation(kind, gate)[0]
    return y if residual is None else _f64(residual) + y


def norm_out_backward(o, weight, dy, gate=None, kind="silu", scale=1.0, eps=1e-6):
    o, w, dz = np.swapaxes(_f64(o), 1, 2), _f64(weight), scale * _f64(dy)
    r = 1.0 / np.sqrt(np.mean(o * o, -1, keepdims=True) + eps)
    n, out = r * o, {}
    if gate is not None:
        act, slope = activation(kind, gate)
        out["dgate"] = dz * w * n * slope
        dz = dz * act
    out["dweight"] = np.sum(dz * n, axis=(0, 1, 2))
    dn = dz * w
    out["dO"] = np.swapaxes(r * (dn - n * np.mean(n * dn, -1, keepdims=True)), 1, 2)
    return out
