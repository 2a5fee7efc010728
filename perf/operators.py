"""Cases and plain forms of the gated linear recurrence and of the norms around a
fast-weight block.

A block of this library runs, between two projections,
  norm_in     token-major q, k, v of the projection -> unit q and k, head-major
  the update  falcon's own rules, or the gated recurrence S_t = a_t S_{t-1} + v_t k_t^T,
              o_t = S_t q_t, a_t = exp(log_a_t)
  norm_out    y = residual + scale * act(gate) * weight * o / rms(o), token-major
`run` computes one of them, forward, backward or for a single token: in elementary torch
operations, or (`own`) through the library's entry points.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_DIMS = (16, 32, 64, 128)


def listed():
    return [
        # a training batch of a 12-head model, 64 dims per head
        dict(name="gated_train", op="gated_fwd", B=8, H=12, L=2048, dk=64, dv=64, dtype="bf16",
             start=False, resets=False),
        # one long document read on from a carried state, few heads, documents' ends inside
        dict(name="gated_long", op="gated_fwd", B=1, H=4, L=32771, dk=128, dv=128, dtype="bf16",
             start=True, resets=True),
        # a short prompt in float32, unequal key and value sizes: latency
        dict(name="gated_short", op="gated_fwd", B=2, H=3, L=77, dk=16, dv=64, dtype="f32",
             start=False, resets=False),
        # gradients of the training batch
        dict(name="gated_train_bwd", op="gated_bwd", B=8, H=12, L=2048, dk=64, dv=64, dtype="bf16",
             start=False, resets=True),
        # truncated training over a long ragged piece: the carried state has a gradient too
        dict(name="gated_long_bwd", op="gated_bwd", B=1, H=5, L=4099, dk=128, dv=64, dtype="bf16",
             start=True, resets=False),
        # serving: 512 sequences x 12 heads, one token each
        dict(name="gated_decode", op="gated_decode", B=512, H=12, L=1, dk=64, dv=64, dtype="bf16",
             start=True, resets=False),
        # serving one sequence: latency
        dict(name="gated_decode_one", op="gated_decode", B=1, H=12, L=1, dk=128, dv=128,
             dtype="bf16", start=True, resets=False),
        # the training batch's projections, views of one fused projection
        dict(name="norm_in_train", op="norm_in", B=8, H=12, L=2048, dk=64, dv=64, dtype="bf16"),
        # its gradient at 128 dims per head, an odd length
        dict(name="norm_in_bwd", op="norm_in_bwd", B=4, H=16, L=1999, dk=128, dv=128,
             dtype="bf16"),
        # serving: the read of 512 sequences' single tokens, gated, into the output projection
        dict(name="norm_out_serve", op="norm_out", B=512, H=12, L=1, dk=64, dv=64, dtype="bf16",
             gate="silu", residual=False),
        # the training batch, added to the residual stream
        dict(name="norm_out_train", op="norm_out", B=8, H=12, L=2048, dk=64, dv=64, dtype="bf16",
             gate="silu", residual=True),
        # the gradient of a long batch at 128 dims per head
        dict(name="norm_out_bwd", op="norm_out_bwd", B=2, H=16, L=8192, dk=128, dv=128,
             dtype="bf16", gate="sigmoid", residual=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_fwd", "gated_bwd", "gated_bwd", "gated_decode", "norm_in",
                     "norm_in_bwd", "norm_out", "norm_out_bwd"])
    c = dict(op=op, H=rng.randint(1, 16), dk=rng.choice(_DIMS), dv=rng.choice(_DIMS),
             dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    d = max(c["dk"], c["dv"])
    if op == "gated_decode":
        c["L"] = 1
        c["B"] = _log_int(rng, 1, max(1, min(768, 512 * 12 * 64 * 64 // (c["H"] * c["dk"] * c["dv"]))))
    else:
        # tokens x heads x dims up to the largest listed cases'
        most = {"gated_fwd": 8 * 12 * 2048 * 64, "gated_bwd": 5 * 4099 * 128}.get(op, 8 * 12 * 2048 * 64)
        if c["dtype"] == "f32":
            most //= 2
        c["L"] = _log_int(rng, 1, max(1, min(16384, most // (c["H"] * d))))
        c["B"] = _log_int(rng, 1, max(1, min(64, most // (c["H"] * d * c["L"]))))
    if op.startswith("gated"):
        c["start"] = op == "gated_decode" or rng.random() < 0.5
        c["resets"] = rng.random() < 0.4
    if op.startswith("norm_out"):
        c["gate"] = rng.choice(["silu", "sigmoid", "none"])
        c["residual"] = op == "norm_out" and rng.random() < 0.5
    return c


def work(case):
    B, H, L, dk, dv = (case[n] for n in ("B", "H", "L", "dk", "dv"))
    es = 2 if case["dtype"] == "bf16" else 4
    n, s, op = B * H * L, B * H * dk * dv * 4, case["op"]
    qkv = (2 * dk + dv) * es
    if op == "gated_fwd":       # q, k, v, log_a in; o out; the states in and out
        return dict(bytes=n * (qkv + 4 + 4 * dv) + s * (2 if case["start"] else 1),
                    flops=4 * n * dk * dv)
    if op == "gated_bwd":       # also dO in; dq, dk, dv, dlog_a out
        return dict(bytes=n * (qkv + 4 + 4 * dv + 4 * (2 * dk + dv) + 4)
                    + s * (3 if case["start"] else 1), flops=12 * n * dk * dv)
    if op == "gated_decode":
        return dict(bytes=2 * s + n * (qkv + 4 + 4 * dv), flops=4 * n * dk * dv)
    if op == "norm_in":
        return dict(bytes=2 * n * qkv, flops=n * (8 * dk))
    if op == "norm_in_bwd":
        return dict(bytes=n * (2 * dk * es + 4 * (2 * dk + dv) + qkv), flops=n * (14 * dk + dv))
    g = dv * es if case["gate"] != "none" else 0
    if op == "norm_out":
        return dict(bytes=n * (4 * dv + g + dv * es + (dv * es if case["residual"] else 0)),
                    flops=12 * n * dv)
    return dict(bytes=n * (4 * dv + 2 * g + dv * es + 4 * dv), flops=24 * n * dv)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).add(1e-12).sqrt()


def prepare(case, seed):
    """Inputs on the GPU: unit q and k and N(0,1) v for the recurrence, gates between about
    0.8 and 0.999 as a sigmoid with a positive bias gives them (resets: about one token in
    300 starts a new document, log_a = -inf); projections of N(0,1) entries for the norms."""
    g, T = _gen(seed), _TYPES[case["dtype"]]
    B, H, L, dk, dv, op = (case[n] for n in ("B", "H", "L", "dk", "dv", "op"))

    def rn(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    s = dict(case=dict(case))
    if op.startswith("gated"):
        lead = (B, H) if op == "gated_decode" else (B, H, L)
        s["q"], s["k"] = _unit(rn(*lead, dk)).to(T), _unit(rn(*lead, dk)).to(T)
        s["v"] = rn(*lead, dv).to(T)
        s["log_a"] = torch.nn.functional.logsigmoid(rn(*lead, std=1.5) + 4.0)
        if case["resets"]:
            s["log_a"][torch.rand(lead, generator=g, device="cuda") < 1 / 300] = -math.inf
        s["S0"] = rn(B, H, dv, dk, std=0.3) if case["start"] else None
        if op == "gated_bwd":
            s["dO"] = rn(B, H, L, dv)
            s["dS_L"] = rn(B, H, dv, dk, std=0.3) if case["start"] else None
    elif op.startswith("norm_in"):
        # one fused projection [B, L, H*dk + H*dk + H*dv]; q, k, v are views of it
        p = rn(B, L, H * (2 * dk + dv)).to(T)
        s["q_in"] = p[..., :H * dk].view(B, L, H, dk)
        s["k_in"] = p[..., H * dk:2 * H * dk].view(B, L, H, dk)
        s["v_in"] = p[..., 2 * H * dk:].view(B, L, H, dv)
        if op == "norm_in_bwd":
            s["dq"], s["dk"], s["dv"] = rn(B, H, L, dk), rn(B, H, L, dk), rn(B, H, L, dv)
    else:
        s["o"] = rn(B, H, L, dv, std=0.5)
        s["weight"] = 1.0 + rn(dv, std=0.1)
        s["gate"] = rn(B, L, H, dv).to(T) if case["gate"] != "none" else None
        s["residual"] = rn(B, L, H, dv).to(T) if case["residual"] else None
        s["scale"] = 0.5
        if op == "norm_out_bwd":
            s["dy"] = rn(B, L, H, dv).to(T)
    return s


# ------------------------------------------------------------- plain forms

_CHUNK = 64


def _chunks(x, n):
    """[B, H, L, ...] -> [B, H, n, 64, ...], zeros behind the last token."""
    pad = n * _CHUNK - x.shape[2]
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[:2] + (pad,) + x.shape[3:])], 2)
    return x.reshape(x.shape[:2] + (n, _CHUNK) + x.shape[3:])


def _decays(x, keep):
    """exp of log decays held in 64 bits, in 32 bits; zero where not kept."""
    return x.masked_fill(~keep, -math.inf).exp().float()


def _gated_plain(q, k, v, log_a, S0):
    """The recurrence in chunks of 64 tokens, all in float32 but the sums of log decays."""
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    n = -(-L // _CHUNK)
    dev = q.device
    # e^-1000 is 0 in 32 bits: a reset's sum of log decays stays finite
    G = _chunks(log_a.double().clamp(min=-1000.0), n).cumsum(-1)
    q, k, v = _chunks(q, n), _chunks(k, n), _chunks(v, n)
    i = torch.arange(_CHUNK, device=dev)
    D = _decays(G[..., :, None] - G[..., None, :], i[:, None] >= i[None, :])
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * D, v)
    # each chunk's own write to the state, and the states that the chunks start from
    total = G[..., -1]
    kv = torch.matmul((v * (total[..., None] - G).exp().float()[..., None]).transpose(-1, -2), k)
    T = torch.cat([total.new_zeros(B, H, 1), total.cumsum(-1)], -1)
    j = torch.arange(n + 1, device=dev)
    W = _decays(T[..., :, None] - T[..., None, 1:], j[:, None] > j[None, :n])
    S = torch.matmul(W, kv.reshape(B, H, n, dv * dk))
    if S0 is not None:
        S = S + T.exp().float()[..., None] * S0.reshape(B, H, 1, dv * dk)
    S = S.reshape(B, H, n + 1, dv, dk)
    o = o + G.exp().float()[..., None] * torch.matmul(q, S[:, :, :n].transpose(-1, -2))
    return o.reshape(B, H, n * _CHUNK, dv)[:, :, :L], S[:, :, n]


def _act(kind, g):
    """act(g) and its derivative."""
    s = 1.0 / (1.0 + torch.exp(-g))
    return (s, s * (1.0 - s)) if kind == "sigmoid" else (g * s, s * (1.0 + g * (1.0 - s)))


def _heads_first(x):
    return x.transpose(1, 2)


def _run_plain(s):
    c, f = s["case"], torch.float32
    op, T = c["op"], _TYPES[c["dtype"]]
    if op == "gated_fwd":
        o, S = _gated_plain(s["q"].to(f), s["k"].to(f), s["v"].to(f), s["log_a"], s["S0"])
        return dict(o=o.contiguous(), S=S.contiguous())
    if op == "gated_bwd":
        with torch.enable_grad():
            x = [s[n].to(f).detach().requires_grad_() for n in ("q", "k", "v", "log_a")]
            x += [s["S0"].detach().requires_grad_()] if s["S0"] is not None else []
            o, S = _gated_plain(*x[:4], x[4] if len(x) == 5 else None)
            loss = (o * s["dO"]).sum() + (0.0 if s["dS_L"] is None else (S * s["dS_L"]).sum())
            d = torch.autograd.grad(loss, x)
        out = dict(zip(("dq", "dk", "dv", "dlog_a", "dS0"), d))
        return out
    if op == "gated_decode":
        a = s["log_a"].exp()[..., None, None]
        v, k = s["v"].to(f), s["k"].to(f)
        s["S0"].mul_(a).add_(v[..., :, None] * k[..., None, :])
        o = (s["S0"] * s["q"].to(f)[..., None, :]).sum(-1)
        return dict(o=o, S=s["S0"])
    if op == "norm_in":
        q, k, v = (_heads_first(s[n].to(f)) for n in ("q_in", "k_in", "v_in"))
        q = q * torch.rsqrt(q.square().sum(-1, keepdim=True) + 1e-6)
        k = k * torch.rsqrt(k.square().sum(-1, keepdim=True) + 1e-6)
        return dict(q=q.to(T).contiguous(), k=k.to(T).contiguous(), v=v.to(T).contiguous())
    if op == "norm_in_bwd":
        def back(x, dy):
            x, dy = x.to(f), _heads_first(dy)
            r = torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)
            y = x * r
            return (r * (dy - y * (y * dy).sum(-1, keepdim=True))).to(T).contiguous()
        return dict(dq_in=back(s["q_in"], s["dq"]), dk_in=back(s["k_in"], s["dk"]),
                    dv_in=_heads_first(s["dv"]).to(T).contiguous())
    o, w = _heads_first(s["o"]), s["weight"]
    r = torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-6)
    if op == "norm_out":
        y = o * r * w
        if s["gate"] is not None:
            y = y * _act(c["gate"], s["gate"].to(f))[0]
        y = y * s["scale"]
        if s["residual"] is not None:
            y = s["residual"].to(f) + y
        return dict(y=y.to(T).contiguous())
    n, dz, out = o * r, s["dy"].to(f) * s["scale"], {}
    if s["gate"] is not None:
        a, da = _act(c["gate"], s["gate"].to(f))
        out["dgate"] = (dz * n * w * da).to(T).contiguous()
        dz = dz * a
    out["dweight"] = (dz * n).sum((0, 1, 2))
    dn = dz * w
    out["dO"] = _heads_first(r * (dn - n * (n * dn).mean(-1, keepdim=True))).contiguous()
    return out


# ------------------------------------------------------- the library's calls

def _run_own(s):
    import weight_recurrent_memory_amd as fw
    c = s["case"]
    op = c["op"]
    if op == "gated_fwd":
        o, S = fw.gated_fwd_chunk(s["q"], s["k"], s["v"], s["log_a"], S0=s["S0"],
                                  return_state=True)
        return dict(o=o, S=S)
    if op == "gated_bwd":
        return fw.gated_bwd_chunk(s["q"], s["k"], s["v"], s["log_a"], s["dO"], S0=s["S0"],
                                  dS_L=s["dS_L"])
    if op == "gated_decode":
        o = fw.gated_decode_step(s["S0"], s["q"], s["k"], s["v"], s["log_a"])
        return dict(o=o, S=s["S0"])
    if op == "norm_in":
        q, k, v = fw.norm_in(s["q_in"], s["k_in"], s["v_in"], eps=1e-6)
        return dict(q=q, k=k, v=v)
    if op == "norm_in_bwd":
        dq, dk, dv = fw.norm_in_bwd(s["q_in"], s["k_in"], s["dq"], s["dk"], s["dv"], eps=1e-6)
        return dict(dq_in=dq, dk_in=dk, dv_in=dv)
    kind = "silu" if c["gate"] == "none" else c["gate"]
    if op == "norm_out":
        return dict(y=fw.norm_out(s["o"], s["weight"], s["gate"], gate_kind=kind,
                                  residual=s["residual"], scale=s["scale"], eps=1e-6,
                                  dtype=_TYPES[c["dtype"]]))
    return fw.norm_out_bwd(s["o"], s["weight"], s["dy"], s["gate"], gate_kind=kind,
                           scale=s["scale"], eps=1e-6)


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions in float64: the recurrence one token at a time."""
    s = prepare(case, seed)
    op, f = case["op"], torch.float64
    x = {n: t.to(f) for n, t in s.items() if isinstance(t, torch.Tensor)}
    if op in ("gated_fwd", "gated_bwd", "gated_decode"):
        return _exact_gated(case, x)
    if op == "norm_in":
        unit = lambda t: (t / (t.pow(2).sum(-1, keepdim=True) + 1e-6).pow(0.5)).permute(0, 2, 1, 3)  # noqa: E731
        return dict(q=unit(x["q_in"]), k=unit(x["k_in"]), v=x["v_in"].permute(0, 2, 1, 3))
    if op == "norm_in_bwd":
        def jacobian(t, dy):
            n2 = t.pow(2).sum(-1, keepdim=True) + 1e-6
            dy = dy.permute(0, 2, 1, 3)
            return dy / n2.pow(0.5) - t * (t * dy).sum(-1, keepdim=True) / n2.pow(1.5)
        return dict(dq_in=jacobian(x["q_in"], x["dq"]), dk_in=jacobian(x["k_in"], x["dk"]),
                    dv_in=x["dv"].permute(0, 2, 1, 3))
    o, w, dv = x["o"], x["weight"], case["dv"]
    gate = x["gate"].permute(0, 2, 1, 3) if "gate" in x else None
    rms = (o.pow(2).sum(-1, keepdim=True) / dv + 1e-6).pow(0.5)
    if gate is None:
        act, slope = torch.ones_like(o), None
    else:
        sg = torch.sigmoid(gate)
        act = sg if case["gate"] == "sigmoid" else gate * sg
        slope = sg * torch.sigmoid(-gate)
        slope = slope if case["gate"] == "sigmoid" else sg + gate * slope
    if op == "norm_out":
        y = (s["scale"] * act * w * o / rms).permute(0, 2, 1, 3)
        return dict(y=y + x["residual"] if "residual" in x else y)
    dy = s["scale"] * x["dy"].permute(0, 2, 1, 3)
    out = dict(dweight=(dy * act * o / rms).reshape(-1, dv).sum(0))
    u = dy * act * w
    out["dO"] = u / rms - o * (u * o).sum(-1, keepdim=True) / (dv * rms.pow(3))
    if gate is not None:
        out["dgate"] = (dy * w * o / rms * slope).permute(0, 2, 1, 3)
    return out


def _exact_gated(case, x):
    B, H, L, dk, dv = (case[n] for n in ("B", "H", "L", "dk", "dv"))
    # [tokens, chains, d]
    q, k, v = (x[n].reshape(B * H, L, -1).transpose(0, 1) for n in ("q", "k", "v"))
    a = x["log_a"].reshape(B * H, L).t().exp()
    S = x["S0"].reshape(B * H, dv, dk) if "S0" in x else q.new_zeros(B * H, dv, dk)
    back = case["op"] == "gated_bwd"
    if back and (L + 1) * S.numel() * 8 > 24e9:
        return None
    states, outs = [S], []
    for t in range(L):
        S = a[t, :, None, None] * S + v[t, :, :, None] * k[t, :, None, :]
        if back:
            states.append(S)
        else:
            outs.append((S * q[t, :, None, :]).sum(-1))
    if not back:
        o = torch.stack(outs, 1)
        return dict(o=o.reshape((B, H, dv) if case["op"] == "gated_decode" else (B, H, L, dv)),
                    S=S.reshape(B, H, dv, dk))
    dO = x["dO"].reshape(B * H, L, dv).transpose(0, 1)
    R = x["dS_L"].reshape(B * H, dv, dk).clone() if "dS_L" in x else torch.zeros_like(S)
    dq, dkk, dvv, dg = [], [], [], []
    for t in range(L - 1, -1, -1):
        R = R + dO[t, :, :, None] * q[t, :, None, :]
        dq.append((states[t + 1] * dO[t, :, :, None]).sum(1))
        dkk.append((R * v[t, :, :, None]).sum(1))
        dvv.append((R * k[t, :, None, :]).sum(2))
        R = a[t, :, None, None] * R
        dg.append((R * states[t]).sum((1, 2)))
    whole = lambda r, *d: torch.stack(r[::-1], 1).reshape((B, H, L) + d)  # noqa: E731
    out = dict(dq=whole(dq, dk), dk=whole(dkk, dk), dv=whole(dvv, dv), dlog_a=whole(dg))
    if "S0" in x:
        out["dS0"] = R.reshape(B, H, dv, dk)
    return out
