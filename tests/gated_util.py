"""For the tests of the gated recurrence: how a call is cut (a mirror of the library's plans,
checked against its workspace sizes), the recurrence and its gradients in float64 on any
device, and the precision that is asked of a whole output.

Bounds of ||error|| / ||output||, u = 2^-24.  A term of an output takes the planes' dropped
parts (three of u), the rounded decay (4u) and a rounded score or state (u), and passes about
30 float32 additions on the matrix cores; roundings point either way, so that they add up as
a root of squares: sqrt(3 + 16 + 1 + 30) < 8u of the terms, whose own root of squares is the
output's size where they are of either sign.  Twice that is asked for: FORWARD = 16u.  A
gradient passes both directions' states: twice as much again.  A third plane left out leaves
up to 2^-17 of every score and state, about 40u of an output (tests/test_gated_plans.py shows
both on the CPU).
"""
import numpy as np

U = 2.0 ** -24
FORWARD, GRADIENT = 16 * U, 32 * U
C = 64
DIMS = (16, 32, 64, 128)


# -------------------------------------------------------------------- plans

def _chunks(L):
    return (L + C - 1) // C


def _cut(units, L, slots, most, whole):
    """(segments, chunks of one)."""
    n = slots // units if units < slots and _chunks(L) >= whole else 1
    n = min(n, max(_chunks(L) // 2, 1))
    per = min((_chunks(L) + n - 1) // n, most)
    return (_chunks(L) + per - 1) // per, per


def _rows_of(nz, chains, L, whole):
    segs = _chunks(L) // 2 if _chunks(L) >= whole else 1
    rows = min(nz, 64)
    while rows > 16 and chains * segs * (nz // rows) < 256:
        rows //= 2
    return rows


def _span_bytes(writes, chains, state):
    return (chains * ((writes + 1) * state + writes) + 3) // 4 * 16 if writes else 0


def forward_plan(chains, L, dk, dv, f32):
    """Value rows of a workgroup, segments, workspace bytes."""
    block = _rows_of(dv, chains, L, 13)
    held = (2 if dk <= 64 else 1) if f32 else (3 if dk <= 64 else 2)
    segs, _ = _cut(chains * (dv // block), L, 256 * held, 1 << 40, 13)
    return block, segs, _span_bytes(segs - 1, chains, dv * dk)


def backward_plan(chains, L, dk, dv, f32):
    """Columns of a workgroup (0: all, up to 64), segments, workspace bytes (with gates
    and an end's gradient)."""
    wide = max(dk, dv) > 64
    most = 32 if not f32 and dk >= 64 else 64
    block_for = lambda whole: min(_rows_of(128, chains, L, whole), most)  # noqa: E731
    whole, walks = (8 if wide else 5), 2 * chains
    if wide:
        b = block_for(1 << 40)
        walks = chains * (2 * -(-dk // b) + -(-dv // b))
    if walks >= 192:
        whole = 17 if walks >= 320 else 13
    block = block_for(whole) if wide else 0
    blocks = dk // block if block and block < dk else 1
    segs, _ = _cut(chains * blocks, L, 512, 16, whole)
    spans = _span_bytes(segs, chains, dv * dk) + _span_bytes(segs - 1, chains, dv * dk)
    return block, segs, spans + 8 * blocks * chains * L


# Cases that reach every kernel: (f32, dk, dv, chains, L)
FORWARD_CASES = [(f32, dk, dv, chains, L) for f32 in (False, True) for dk in DIMS
                 for dv, chains, L in ((16, 3, 130), (64, 128, 130), (128, 128, 65),       # whole
                                       (64, 3, 850), (64, 19, 850), (128, 19, 833))]       # cut
BACKWARD_CASES = [(f32, dk, dv, 3, L) for f32 in (False, True) for dk in DIMS[:3] for dv in DIMS[:3]
                  for L in (130, 400)]
BACKWARD_CASES += [(f32, dk, dv, chains, L) for f32 in (False, True) for dk in DIMS for dv in DIMS
                   if max(dk, dv) == 128
                   for chains, L in ((3, 130), (64, 130), (128, 65), (3, 600), (8, 1090), (15, 1090))
                   # (more chains take no larger blocks there)
                   if f32 or dk < 64 or chains not in (128, 15)]


# ------------------------------------------------- the definitions, float64

def recurrence(torch, q, k, v, log_a, S0):
    """o, S_L and the states S_0 .. S_L; torch tensors, any float type."""
    q, k, v = q.double(), k.double(), v.double()
    B, H, L, dk = q.shape
    a = torch.ones(B, H, L, dtype=torch.float64, device=q.device) if log_a is None else log_a.double().exp()
    S = q.new_zeros(B, H, v.shape[-1], dk) if S0 is None else S0.double()
    states, o = [S], []
    for t in range(L):
        S = a[:, :, t, None, None] * S + v[:, :, t, :, None] * k[:, :, t, None, :]
        states.append(S)
        o.append((S * q[:, :, t, None, :]).sum(-1))
    return torch.stack(o, 2), S, states


def gradients(torch, q, k, v, log_a, S0, dO, dS_L):
    states = recurrence(torch, q, k, v, log_a, S0)[2]
    q, k, v, dO = q.double(), k.double(), v.double(), dO.double()
    L = q.shape[2]
    a = torch.ones_like(q[..., 0]) if log_a is None else log_a.double().exp()
    R = torch.zeros_like(states[0]) if dS_L is None else dS_L.double()
    dq, dkk, dvv, dg = [], [], [], []
    for t in range(L - 1, -1, -1):
        R = R + dO[:, :, t, :, None] * q[:, :, t, None, :]
        dq.append((states[t + 1] * dO[:, :, t, :, None]).sum(-2))
        dkk.append((R * v[:, :, t, :, None]).sum(-2))
        dvv.append((R * k[:, :, t, None, :]).sum(-1))
        R = a[:, :, t, None, None] * R
        dg.append((R * states[t]).sum((-1, -2)))
    whole = lambda x: torch.stack(x[::-1], 2)  # noqa: E731
    return dict(dq=whole(dq), dk=whole(dkk), dv=whole(dvv), dlog_a=whole(dg), dS0=R)


def off(got, want):
    """||got - want|| / ||want||."""
    got, want = (np.asarray(x.detach().cpu() if hasattr(x, "detach") else x, dtype=np.float64)
                 for x in (got, want))
    return float(np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-300))
