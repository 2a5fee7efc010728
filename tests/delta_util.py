"""For the tests of the gated delta rule: inputs, the rule and its gradients in float64 on any
device, and the precision that is asked of a whole output.

Bounds of ||error|| / ||output||, u = 2^-24, for unit keys and 0 <= beta <= 2, where no token's
factor a (I - beta k k^T) is larger than one and an error does not grow.  An output passes three
products one behind the other (keys with the state, T with what they leave, scores or keys with
u); each takes the planes' dropped parts (three of u), rounded decays (4u), a rounded operand (u)
and about 30 float32 additions: sqrt(3 + 16 + 1 + 30) < 8u of its terms, as roundings point
either way.  T itself is three such products of blocks.  sqrt(6) 8u < 20u where the terms are of
the output's own size; FORWARD = 40u asks for twice that.  A gradient passes both directions'
walks: GRADIENT = 80u.
"""
import numpy as np

U = 2.0 ** -24
FORWARD, GRADIENT = 40 * U, 80 * U
DIMS = (16, 32, 64, 128)


def inputs(torch, seed, B, H, L, dk, dv, dtype, *, gate="mixed", start=True, beta="mixed", keys="random",
           device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=g, device=device)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=unit(rn(B, H, L, dk)).to(dtype), k=unit(rn(B, H, L, dk)), v=rn(B, H, L, dv).to(dtype))
    if keys == "repeated":               # long runs of one key
        x["k"] = x["k"][:, :, torch.arange(L, device=device) // 40 * 40]
    x["k"] = x["k"].to(dtype)
    x["beta"] = dict(mixed=torch.sigmoid(1.5 * rn(B, H, L)), one=torch.ones(B, H, L, device=device),
                     zero=(rand(B, H, L) < 0.5).float(), two=2.0 * rand(B, H, L))[beta]
    log_a = torch.nn.functional.logsigmoid(2.0 * rn(B, H, L) + 3.0)
    if gate == "strong":                 # decays down to e^-60 beside weak ones
        log_a = torch.where(rand(B, H, L) < 0.3, -60 * rand(B, H, L), log_a)
    if gate == "resets":
        log_a = torch.where(rand(B, H, L) < 0.05, torch.full_like(log_a, -float("inf")), log_a)
    x["log_a"] = None if gate == "none" else log_a
    x["S0"] = 0.3 * rn(B, H, dv, dk) if start else None
    x["dO"], x["dS_L"] = rn(B, H, L, dv), 0.3 * rn(B, H, dv, dk)
    return x


def recurrence(torch, x):
    """o, S_L, the states S_0 .. S_L and what u is of beta."""
    q, k, v, b = (x[n].double() for n in ("q", "k", "v", "beta"))
    B, H, L, dk = q.shape
    a = torch.ones_like(b) if x["log_a"] is None else x["log_a"].double().exp()
    S = q.new_zeros(B, H, v.shape[-1], dk) if x["S0"] is None else x["S0"].double()
    states, o, errs = [S], [], []
    for t in range(L):
        S = a[:, :, t, None, None] * S
        errs.append(v[:, :, t] - (S * k[:, :, t, None, :]).sum(-1))
        S = S + (b[:, :, t, None] * errs[-1])[..., None] * k[:, :, t, None, :]
        states.append(S)
        o.append((S * q[:, :, t, None, :]).sum(-1))
    return torch.stack(o, 2), S, states, errs


def gradients(torch, x, dS_L=True):
    _, S, states, errs = recurrence(torch, x)
    q, k, b, dO = (x[n].double() for n in ("q", "k", "beta", "dO"))
    L = q.shape[2]
    a = torch.ones_like(b) if x["log_a"] is None else x["log_a"].double().exp()
    R = x["dS_L"].double() if dS_L else torch.zeros_like(S)
    out = dict(dq=[], dk=[], dv=[], dbeta=[], dlog_a=[])
    for t in range(L - 1, -1, -1):
        bt = b[:, :, t, None]
        R = R + dO[:, :, t, :, None] * q[:, :, t, None, :]
        before = a[:, :, t, None, None] * states[t]
        du = (R * k[:, :, t, None, :]).sum(-1)
        out["dq"].append((states[t + 1] * dO[:, :, t, :, None]).sum(-2))
        out["dk"].append(bt * ((R * errs[t][..., None]).sum(-2) - (before * du[..., None]).sum(-2)))
        out["dv"].append(bt * du)
        out["dbeta"].append((du * errs[t]).sum(-1))
        R = R - (bt * du)[..., None] * k[:, :, t, None, :]
        out["dlog_a"].append((R * before).sum((-1, -2)))
        R = a[:, :, t, None, None] * R
    out = {n: torch.stack(y[::-1], 2) for n, y in out.items()}
    out["dS0"] = R
    return out


C, SLOTS, GAIN, XCDS = 64, 256, 6, 8


def write_blocks(rows):
    """Workgroups of four waves for so many rows of a segment's own write and matrix."""
    return -(-rows // 64)


def _ahead(dk, f32):
    return 2 if not f32 and dk <= 64 else 1


def key_lds(dk, f32):
    """LDS of a workgroup without outputs: a chunk's keys and gates, one or two ahead, and two T."""
    return (_ahead(dk, f32) + 1) * ((3 if f32 else 1) * C * dk * 2 + 1552) + 16 + 2 * 18432


def walk_lds(dk, f32, waves):
    """The forward's main walk: S's and u's operands of two chunks in place of T."""
    s, u = -(-dk // 32) * 3, 6 if dk == 128 else 4
    return key_lds(dk, f32) - 2 * 18432 + 2 * waves * (s + u) * 1024


def rounds(blocks, lds, segments):
    """Rounds of a launch of so many workgroups a segment, a segment's on one XCD of 32 compute units."""
    return -(-(-(-segments // XCDS) * blocks) // (SLOTS // XCDS * (2 if 2 * lds <= 163840 else 1)))


def cut(chunks, chains, write, unwritten, walk, dk):
    """Segments of a chain; write and walk: workgroups a segment and their LDS."""
    n = min(SLOTS // (chains * write[0]), chunks // 2)
    if n < 2:
        return 1
    each = -(-chunks // n)
    n = -(-chunks // each)
    first = rounds(*write, chains * (n - unwritten)) if dk < 128 else 1
    if each * (first + rounds(*walk, chains * n)) + GAIN > chunks * rounds(*walk, chains):
        return 1
    return n


def _segments(chains, segs, dk, dv):
    return chains * segs * (dv * dk * 4 + dk // 16 * ((dk + 31) // 32) * 3 * 64 * 16) if segs > 1 else 0


def forward_plan(chains, L, dk, dv, f32):
    """(state waves of a workgroup of the main walk, segments of a chain, bytes of workspace)."""
    chunks = -(-L // C)
    waves = 1 if dv == 16 or (f32 and dk == 128) else 2
    segs = cut(chunks, chains, (write_blocks(dv + dk), key_lds(dk, f32)), 1,
               (dv // (16 * waves), walk_lds(dk, f32, waves)), dk)
    return waves, segs, chains * chunks * 18432 + _segments(chains, segs, dk, dv)


def backward_plan(chains, L, dk, dv, f32):
    """(state waves of a workgroup of the main walks, segments of a chain, bytes of workspace)."""
    chunks = -(-L // C)
    waves, lds = min(dv // 16, 4), key_lds(dk, f32)
    segs = cut(chunks, chains, (write_blocks(dv + dk) + write_blocks(dv), lds), 0, (2 * (dv // (16 * waves)), lds), dk)
    chunk = 2 * 18432 + C * dv * 4 + 3 * dv * dk * 4
    return waves, segs, chains * (chunks * chunk + L * dv * 4) + 2 * _segments(chains, segs, dk, dv)


# (f32, dk, dv, chains, L): every size in both types, walked whole and cut
PLAN_CASES = [(f32, dk, dv, 2, L) for f32 in (False, True) for dk in DIMS for dv in DIMS for L in (150, 1030)]


def norm(x):
    return float(np.linalg.norm(np.asarray(x.detach().cpu(), dtype=np.float64)))


def off(got, want):
    """||got - want|| / ||want||."""
    assert got.shape == want.shape
    return norm(got.double() - want) / max(norm(want), 1e-300)
