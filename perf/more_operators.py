"""Cases and plain forms of the gated delta rule and of rotary positions at a fast-weight
block's entry.

  gated_delta  S_t = a_t S_{t-1} + u_t k_t^T,  u_t = beta_t (v_t - a_t S_{t-1} k_t),
               o_t = S_t q_t,  a_t = exp(log_a_t): forward, backward, one token
  rotary_in    token-major q, k, v of a projection -> unit q and k, turned by their
               positions, head-major: forward and backward
`run` computes one of them in elementary torch operations, or (`own`) through the
library's entry points.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_DIMS = (16, 32, 64, 128)


def listed():
    return [
        # a training batch of a 12-head model, 64 dims per head
        dict(name="delta_train", op="delta_fwd", B=8, H=12, L=2048, dk=64, dv=64, dtype="bf16",
             start=False, resets=False),
        # one long document read on from a carried state, few heads, documents' ends inside
        dict(name="delta_long", op="delta_fwd", B=1, H=4, L=32771, dk=128, dv=128, dtype="bf16",
             start=True, resets=True),
        # a short prompt in float32, unequal key and value sizes: latency
        dict(name="delta_short", op="delta_fwd", B=2, H=3, L=77, dk=16, dv=64, dtype="f32",
             start=False, resets=False),
        # gradients of the training batch
        dict(name="delta_train_bwd", op="delta_bwd", B=8, H=12, L=2048, dk=64, dv=64, dtype="bf16",
             start=False, resets=True),
        # truncated training over a long ragged piece: the carried state has a gradient too
        dict(name="delta_long_bwd", op="delta_bwd", B=1, H=5, L=4099, dk=128, dv=64, dtype="bf16",
             start=True, resets=False),
        # gradients of a few short sequences in float32
        dict(name="delta_short_bwd", op="delta_bwd", B=2, H=3, L=130, dk=32, dv=32, dtype="f32",
             start=False, resets=False),
        # serving: 512 sequences x 12 heads, one token each
        dict(name="delta_decode", op="delta_decode", B=512, H=12, L=1, dk=64, dv=64, dtype="bf16",
             start=True, resets=False),
        # serving one sequence: latency
        dict(name="delta_decode_one", op="delta_decode", B=1, H=12, L=1, dk=128, dv=128,
             dtype="bf16", start=True, resets=False),
        # the training batch's projections, views of one fused projection, whole heads turned
        dict(name="rotary_train", op="rotary_in", B=8, H=12, L=2048, dk=64, dv=64, dtype="bf16",
             rot=64, pairs="half", factor=1.0),
        # a long piece of a far document: half of each head turned, neighbours paired, scaled
        # frequencies, float32
        dict(name="rotary_far", op="rotary_in", B=1, H=8, L=8191, dk=128, dv=128, dtype="f32",
             rot=64, pairs="neighbours", factor=8.0),
        # serving: single tokens of 512 sequences, each at a position of its own
        dict(name="rotary_serve", op="rotary_in", B=512, H=12, L=1, dk=64, dv=64, dtype="bf16",
             rot=64, pairs="half", factor=4.0),
        # the gradient at 128 dims per head, an odd length
        dict(name="rotary_bwd", op="rotary_in_bwd", B=4, H=16, L=1999, dk=128, dv=128,
             dtype="bf16", rot=128, pairs="half", factor=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_bwd", "delta_decode", "rotary_in",
                     "rotary_in_bwd"])
    c = dict(op=op, H=rng.randint(1, 16), dk=rng.choice(_DIMS), dv=rng.choice(_DIMS),
             dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    d = max(c["dk"], c["dv"])
    if op == "delta_decode":
        c["L"] = 1
        c["B"] = _log_int(rng, 1, max(1, min(768, 512 * 12 * 64 * 64 // (c["H"] * c["dk"] * c["dv"]))))
    else:
        # tokens x heads x dims up to the largest listed cases'
        most = {"delta_fwd": 8 * 12 * 2048 * 64, "delta_bwd": 5 * 4099 * 128}.get(op, 8 * 12 * 2048 * 64)
        if c["dtype"] == "f32":
            most //= 2
        c["L"] = _log_int(rng, 1, max(1, min(16384, most // (c["H"] * d))))
        c["B"] = _log_int(rng, 1, max(1, min(64, most // (c["H"] * d * c["L"]))))
    if op.startswith("delta"):
        c["start"] = op == "delta_decode" or rng.random() < 0.5
        c["resets"] = rng.random() < 0.4
    else:
        c["rot"] = rng.choice([r for r in (8, 16, 32, 48, 64, 96, 128) if r <= c["dk"]])
        c["pairs"] = rng.choice(["half", "neighbours"])
        c["factor"] = rng.choice([1.0, 1.0, 2.0, 8.0])
    return c


def work(case):
    B, H, L, dk, dv = (case[n] for n in ("B", "H", "L", "dk", "dv"))
    es = 2 if case["dtype"] == "bf16" else 4
    n, s, op = B * H * L, B * H * dk * dv * 4, case["op"]
    qkv = (2 * dk + dv) * es
    if op == "delta_fwd":       # q, k, v, the gates in; o out; the states in and out
        return dict(bytes=n * (qkv + 8 + 4 * dv) + s * (2 if case["start"] else 1),
                    flops=6 * n * dk * dv)
    if op == "delta_bwd":       # also dO in; dq, dk, dv and the gates' gradients out
        return dict(bytes=n * (qkv + 8 + 4 * dv + 4 * (2 * dk + dv) + 8)
                    + s * (3 if case["start"] else 1), flops=18 * n * dk * dv)
    if op == "delta_decode":
        return dict(bytes=2 * s + n * (qkv + 8 + 4 * dv), flops=6 * n * dk * dv)
    positions = 8 * B * L + 4 * case["rot"]
    if op == "rotary_in":
        return dict(bytes=2 * n * qkv + positions, flops=n * 14 * dk)
    return dict(bytes=n * (2 * dk * es + 4 * (2 * dk + dv) + qkv) + positions, flops=n * (20 * dk + dv))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).add(1e-12).sqrt()


def _frequencies(rot, factor):
    """Radians a token of each pair, float64: 10000^(-2i / rot); with a factor, pairs that
    turn less than once over 2048 tokens slowed by it, those that turn 32 times or more left,
    the others in between."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-2.0 * i / rot)
    keep = ((2048.0 * f / (2.0 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * keep + f / factor * (1.0 - keep)


def prepare(case, seed):
    """Inputs on the GPU: unit q and k and N(0,1) v for the recurrence, decays between about
    0.8 and 0.999 and write strengths about one half, both as a sigmoid gives them (resets:
    about one token in 300 starts a new document, log_a = -inf); projections of N(0,1) entries
    and running positions from a start of each sequence's own for the rotation."""
    g, T = _gen(seed), _TYPES[case["dtype"]]
    B, H, L, dk, dv, op = (case[n] for n in ("B", "H", "L", "dk", "dv", "op"))

    def rn(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    s = dict(case=dict(case))
    if op.startswith("delta"):
        lead = (B, H) if op == "delta_decode" else (B, H, L)
        s["q"], s["k"] = _unit(rn(*lead, dk)).to(T), _unit(rn(*lead, dk)).to(T)
        s["v"] = rn(*lead, dv).to(T)
        s["beta"] = torch.sigmoid(rn(*lead, std=1.5))
        s["log_a"] = torch.nn.functional.logsigmoid(rn(*lead, std=1.5) + 4.0)
        if case["resets"]:
            s["log_a"][torch.rand(lead, generator=g, device="cuda") < 1 / 300] = -math.inf
        s["S0"] = rn(B, H, dv, dk, std=0.3) if case["start"] else None
        if op == "delta_bwd":
            s["dO"] = rn(B, H, L, dv)
            s["dS_L"] = rn(B, H, dv, dk, std=0.3) if case["start"] else None
        return s
    # one fused projection [B, L, H*dk + H*dk + H*dv]; q, k, v are views of it
    p = rn(B, L, H * (2 * dk + dv)).to(T)
    s["q_in"] = p[..., :H * dk].view(B, L, H, dk)
    s["k_in"] = p[..., H * dk:2 * H * dk].view(B, L, H, dk)
    s["v_in"] = p[..., 2 * H * dk:].view(B, L, H, dv)
    far = 1000000 if case["factor"] > 1.0 else 4096
    first = torch.randint(0, far, (B, 1), generator=g, device="cuda")
    s["positions"] = first + torch.arange(L, device="cuda")
    s["freqs"] = _frequencies(case["rot"], case["factor"])
    s["scale"] = 0.1 * math.log(case["factor"]) + 1.0
    if op == "rotary_in_bwd":
        s["dq"], s["dk"], s["dv"] = rn(B, H, L, dk), rn(B, H, L, dk), rn(B, H, L, dv)
    return s


# ------------------------------------------------------------- plain forms

_CHUNK = 64


def _chunks(x, n):
    """[B, H, L, ...] -> [n, B, H, 64, ...], zeros behind the last token."""
    pad = n * _CHUNK - x.shape[2]
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[:2] + (pad,) + x.shape[3:])], 2)
    return x.reshape(x.shape[:2] + (n, _CHUNK) + x.shape[3:]).movedim(2, 0)


def _whole(x, L):
    """_chunks' inverse."""
    x = x.movedim(0, 2)
    return x.reshape(x.shape[:2] + (-1,) + x.shape[4:])[:, :, :L].contiguous()


def _t(x):
    return x.transpose(-1, -2)


def _decays(x, keep):
    """exp of log decays held in 64 bits, in 32 bits; zero where not kept."""
    return x.masked_fill(~keep, -math.inf).exp().float()


def _unit_lower_inverse(A):
    """(I + A)^-1 of a strictly lower A, blocks of 1, 2, 4 .. tokens:
    [[X, 0], [C, Y]]^-1 = [[X^-1, 0], [-Y^-1 C X^-1, Y^-1]]."""
    n = A.shape[-1]
    T = torch.eye(n, device=A.device).expand_as(A).contiguous()
    s = 1
    while s < n:
        def blocks(M):
            return M.unflatten(-2, (n // (2 * s), 2 * s)).unflatten(-1, (n // (2 * s), 2 * s)) \
                .diagonal(dim1=-4, dim2=-2)          # [..., 2s, 2s, blocks]
        t, a = blocks(T).movedim(-1, -3), blocks(A).movedim(-1, -3)
        low = -torch.matmul(torch.matmul(t[..., s:, s:], a[..., s:, :s]), t[..., :s, :s])
        blocks(T)[..., s:, :s, :].copy_(low.movedim(-3, -1))
        s *= 2
    return T


def _delta_parts(s):
    """What the chunks need, each [n, B, H, 64, ..]."""
    f, L = torch.float32, s["q"].shape[2]
    n, dev = -(-L // _CHUNK), s["q"].device
    # e^-1000 is 0 in 32 bits: a reset's sum of log decays stays finite
    G = _chunks(s["log_a"].double().clamp(min=-1000.0), n).cumsum(-1)
    x = {m: _chunks(s[m].to(f), n) for m in ("q", "k", "v", "beta")}
    i = torch.arange(_CHUNK, device=dev)
    D = _decays(G[..., :, None] - G[..., None, :], i[:, None] >= i[None, :])
    x["b"] = x["beta"][..., None]
    x["P"] = torch.matmul(x["q"], _t(x["k"])) * D
    x["T"] = _unit_lower_inverse(x["b"] * (torch.matmul(x["k"], _t(x["k"])) * D).tril(-1))
    x["D"] = D
    x["e"] = G.exp().float()[..., None]
    x["w"] = (G[..., -1:] - G).exp().float()[..., None]
    x["d"] = G[..., -1].exp().float()[..., None, None]
    return x


def _delta_forward(x, S0, dv):
    """u and o of every chunk, the states at the chunks' starts and the last one."""
    n, B, H, _, dk = x["k"].shape
    S = x["k"].new_zeros(B, H, dv, dk) if S0 is None else S0
    starts, us = [], []
    for c in range(n):
        starts.append(S)
        u = torch.matmul(x["T"][c], x["b"][c] * (x["v"][c] - x["e"][c] * torch.matmul(x["k"][c], _t(S))))
        us.append(u)
        S = x["d"][c] * S + torch.matmul(_t(u), x["w"][c] * x["k"][c])
    return torch.stack(us), torch.stack(starts), S


def _delta_backward(x, s):
    u, S, S_L = _delta_forward(x, s["S0"], s["v"].shape[-1])
    n = u.shape[0]
    q, k, v, b, e, w, P = (x[m] for m in ("q", "k", "v", "b", "e", "w", "P"))
    dO = _chunks(s["dO"], n)
    R = torch.zeros_like(S_L) if s["dS_L"] is None else s["dS_L"]
    ends, dus = [], []
    for c in range(n - 1, -1, -1):
        ends.append(R)
        du = torch.matmul(_t(x["T"][c]), torch.matmul(_t(P[c]), dO[c]) + w[c] * torch.matmul(k[c], _t(R)))
        dus.append(du)
        R = x["d"][c] * R + torch.matmul(_t(dO[c]), e[c] * q[c]) - torch.matmul(_t(b[c] * du), e[c] * k[c])
    du, ends = torch.stack(dus[::-1]), torch.stack(ends[::-1])
    Z = x["D"] * torch.matmul(dO, _t(u))
    W = (x["D"] * torch.matmul(du, _t(u))).tril(-1)
    dq = e * torch.matmul(dO, S) + torch.matmul(Z, k)
    y = e * torch.matmul(du, S) + torch.matmul(W, k)
    dk = w * torch.matmul(u, ends) + torch.matmul(_t(Z), q) - torch.matmul(_t(b * W), k) - b * y
    dv = b * du
    db = (du * v).sum(-1) - (y * k).sum(-1)
    # what passes each token's border: <R, S> behind the chunk, then token by token
    behind = torch.cat([S[1:], S_L[None]])
    X = (ends.double() * behind).sum((-1, -2))
    step = (q.double() * dq).sum(-1) - (v.double() * dv).sum(-1)
    reset = (_chunks(s["log_a"], n) < -104.0).flip(-1)
    # sums from the chunk's end, begun anew behind a reset
    step = step.flip(-1)
    total = X[..., None] + step.cumsum(-1)
    cut = total.masked_fill(~reset, 0.0)
    i = torch.arange(_CHUNK, device=step.device)
    last = torch.where(reset, i, torch.full_like(i, -1)).cummax(-1).values
    dg = total - torch.where(last >= 0, cut.gather(-1, last.clamp(min=0)), torch.zeros_like(total))
    L = s["q"].shape[2]
    out = dict(dq=dq, dk=dk, dv=dv, dbeta=db, dlog_a=dg.flip(-1).float())
    out = {m: _whole(t, L) for m, t in out.items()}
    if s["S0"] is not None:
        out["dS0"] = R.contiguous()
    return out


def _heads_first(x):
    return x.transpose(1, 2)


def _angles(s):
    """cos and sin of every token's pairs, [B, L, 1, rot / 2], times the scale."""
    a = s["positions"].double()[..., None, None] * s["freqs"]
    return (a.cos() * s["scale"]).float(), (a.sin() * s["scale"]).float()


def _turn(x, cos, sin, rot, pairs):
    """The first rot columns of x turned in pairs."""
    y = x.clone()
    if pairs == "half":
        i, j = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        i, j = slice(0, rot, 2), slice(1, rot, 2)
    y[..., i] = x[..., i] * cos - x[..., j] * sin
    y[..., j] = x[..., j] * cos + x[..., i] * sin
    return y


def _run_plain(s):
    c, f = s["case"], torch.float32
    op, T = c["op"], _TYPES[c["dtype"]]
    if op == "delta_fwd":
        x, L = _delta_parts(s), c["L"]
        u, S, S_L = _delta_forward(x, s["S0"], c["dv"])
        o = x["e"] * torch.matmul(x["q"], _t(S)) + torch.matmul(x["P"], u)
        return dict(o=_whole(o, L), S=S_L.contiguous())
    if op == "delta_bwd":
        return _delta_backward(_delta_parts(s), s)
    if op == "delta_decode":
        q, k, v = (s[m].to(f) for m in ("q", "k", "v"))
        S = s["S0"].mul_(s["log_a"].exp()[..., None, None])
        u = s["beta"][..., None] * (v - (S * k[..., None, :]).sum(-1))
        S.add_(u[..., :, None] * k[..., None, :])
        return dict(o=(S * q[..., None, :]).sum(-1), S=S)
    cos, sin = _angles(s)
    if op == "rotary_in":
        def unit(x):
            x = x.to(f)
            x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)
            return _heads_first(_turn(x, cos, sin, c["rot"], c["pairs"])).to(T).contiguous()
        return dict(q=unit(s["q_in"]), k=unit(s["k_in"]), v=_heads_first(s["v_in"]).contiguous())

    def back(x, dy):
        x, dy = x.to(f), _turn(_heads_first(dy), cos, -sin, c["rot"], c["pairs"])
        r = torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)
        y = x * r
        return (r * (dy - y * (y * dy).sum(-1, keepdim=True))).to(T).contiguous()
    return dict(dq_in=back(s["q_in"], s["dq"]), dk_in=back(s["k_in"], s["dk"]),
                dv_in=_heads_first(s["dv"]).to(T).contiguous())


# ------------------------------------------------------- the library's calls

def _run_own(s):
    import weight_recurrent_memory_amd as fw
    c = s["case"]
    op = c["op"]
    if op == "delta_fwd":
        o, S = fw.gated_delta_fwd_chunk(s["q"], s["k"], s["v"], s["beta"], s["log_a"], S0=s["S0"],
                                        return_state=True)
        return dict(o=o, S=S)
    if op == "delta_bwd":
        return fw.gated_delta_bwd_chunk(s["q"], s["k"], s["v"], s["beta"], s["log_a"], s["dO"],
                                        S0=s["S0"], dS_L=s["dS_L"])
    if op == "delta_decode":
        o = fw.gated_delta_decode_step(s["S0"], s["q"], s["k"], s["v"], s["beta"], s["log_a"])
        return dict(o=o, S=s["S0"])
    if op == "rotary_in":
        q, k, v = fw.rotary_in(s["q_in"], s["k_in"], s["v_in"], s["positions"], s["freqs"],
                               pairs=c["pairs"], scale=s["scale"], eps=1e-6)
        return dict(q=q, k=k, v=v)
    dq, dk, dv = fw.rotary_in_bwd(s["q_in"], s["k_in"], s["dq"], s["dk"], s["dv"], s["positions"],
                                  s["freqs"], pairs=c["pairs"], scale=s["scale"], eps=1e-6)
    return dict(dq_in=dq, dk_in=dk, dv_in=dv)


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions in float64: the recurrence one token at a time."""
    s = prepare(case, seed)
    x = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor)}
    if case["op"].startswith("delta"):
        return _exact_delta(case, x)
    # pairs as complex numbers
    R = case["rot"]
    turn = s["scale"] * torch.polar(torch.ones_like(x["freqs"]) + 0.0 * x["positions"][..., None],
                                    x["positions"][..., None] * x["freqs"])[:, None]

    def pairs_of(t):
        r = t[..., :R]
        r = r.unflatten(-1, (2, R // 2)).transpose(-1, -2) if case["pairs"] == "half" else r.unflatten(-1, (R // 2, 2))
        return torch.view_as_complex(r.contiguous())

    def from_pairs(z, t):
        r = torch.view_as_real(z)
        r = r.transpose(-1, -2) if case["pairs"] == "half" else r
        return torch.cat([r.flatten(-2), t[..., R:]], -1)

    if case["op"] == "rotary_in":
        def out(t):
            t = t.permute(0, 2, 1, 3)
            t = t / (t.pow(2).sum(-1, keepdim=True) + 1e-6).pow(0.5)
            return from_pairs(pairs_of(t) * turn, t)
        return dict(q=out(x["q_in"]), k=out(x["k_in"]), v=x["v_in"].permute(0, 2, 1, 3))

    def jacobian(t, dy):
        dy = from_pairs(pairs_of(dy) * turn.conj(), dy).permute(0, 2, 1, 3)
        n2 = t.pow(2).sum(-1, keepdim=True) + 1e-6
        return dy / n2.pow(0.5) - t * (t * dy).sum(-1, keepdim=True) / n2.pow(1.5)
    return dict(dq_in=jacobian(x["q_in"], x["dq"]), dk_in=jacobian(x["k_in"], x["dk"]),
                dv_in=x["dv"].permute(0, 2, 1, 3))


def _exact_delta(case, x):
    B, H, L, dk, dv = (case[n] for n in ("B", "H", "L", "dk", "dv"))
    # [tokens, chains, d]
    q, k, v = (x[n].reshape(B * H, L, -1).transpose(0, 1).contiguous() for n in ("q", "k", "v"))
    a, b = (t.reshape(B * H, L).t().contiguous() for t in (x["log_a"].exp(), x["beta"]))
    S = x["S0"].reshape(B * H, dv, dk) if "S0" in x else q.new_zeros(B * H, dv, dk)
    back = case["op"] == "delta_bwd"
    if back and (L + 1) * S.numel() * 8 > 24e9:
        return None
    states, outs, errs = [S], [], []
    for t in range(L):
        S = a[t, :, None, None] * S
        r = v[t] - torch.matmul(S, k[t, :, :, None])[..., 0]
        S = torch.baddbmm(S, (b[t, :, None] * r)[:, :, None], k[t, :, None, :])
        if back:
            states.append(S)
            errs.append(r)
        else:
            outs.append(torch.matmul(S, q[t, :, :, None])[..., 0])
    if not back:
        o = torch.stack(outs, 1)
        return dict(o=o.reshape((B, H, dv) if case["op"] == "delta_decode" else (B, H, L, dv)),
                    S=S.reshape(B, H, dv, dk))
    dO = x["dO"].reshape(B * H, L, dv).transpose(0, 1).contiguous()
    R = x["dS_L"].reshape(B * H, dv, dk).clone() if "dS_L" in x else torch.zeros_like(S)
    dq, dkk, dvv, dbb, dg = [], [], [], [], []
    for t in range(L - 1, -1, -1):
        R = torch.baddbmm(R, dO[t, :, :, None], q[t, :, None, :])
        du = torch.matmul(R, k[t, :, :, None])
        before = a[t, :, None, None] * states[t]
        dq.append(torch.matmul(dO[t, :, None, :], states[t + 1])[:, 0])
        dkk.append(b[t, :, None] * (torch.matmul(errs[t][:, None, :], R) - torch.matmul(du.mT, before))[:, 0])
        dvv.append(b[t, :, None] * du[..., 0])
        dbb.append((du[..., 0] * errs[t]).sum(-1))
        R = R - b[t, :, None, None] * du * k[t, :, None, :]
        dg.append((R * before).sum((1, 2)))
        R = a[t, :, None, None] * R
    whole = lambda r, *d: torch.stack(r[::-1], 1).reshape((B, H, L) + d)  # noqa: E731
    out = dict(dq=whole(dq, dk), dk=whole(dkk, dk), dv=whole(dvv, dv), dbeta=whole(dbb), dlog_a=whole(dg))
    if "S0" in x:
        out["dS0"] = R.reshape(B, H, dv, dk)
    return out
