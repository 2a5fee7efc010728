"""The gated recurrence's chunk forward and backward against the fp64 recurrence.

Tolerances, u = 2^-24 (float32).  The oracle is also run on absolute values, which
gives for each output the sum A of the absolute values of its terms.  The kernels form
each term with at most: the planes' dropped parts 3u a product of two products, decays
to 4u (a float32 exponent, v_exp_f32), and float32 sums, at most 64 + dk terms inside a
chunk in matrix-core order and one rounding of the state a chunk while a term lives.  A
worst case of every rounding the same way: (dk + dv + 80 + 8 chunks) u A for the forward;
roundings do not all point one way, so errors stay well below it.  The comparison is per
element with the tensor's rounding floor (A itself is at least a millionth of its mean).
"""
import numpy as np
import pytest

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import weight_recurrent_memory_amd as fw  # noqa: E402

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fw.load_library()


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _up(x, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(dtype)


def _inputs(seed, B, H, L, dk, dv, dtype, *, gate="mixed", start=True):
    r = np.random.default_rng(seed)
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    x = dict(q=_up(unit(n(B, H, L, dk)), dtype), k=_up(unit(n(B, H, L, dk)), dtype),
             v=_up(n(B, H, L, dv), dtype))
    g = -np.log1p(np.exp(-(2.0 * n(B, H, L) + 3.0)))
    if gate == "strong":                 # decays down to e^-60 beside weak ones
        g = np.where(r.random((B, H, L)) < 0.3, -60 * r.random((B, H, L)), g)
    if gate == "resets":
        g = np.where(r.random((B, H, L)) < 0.05, -np.inf, g)
    x["log_a"] = None if gate == "none" else _up(g)
    x["S0"] = _up(0.3 * n(B, H, dv, dk)) if start else None
    return x


def _forward_ref(x):
    a = [_np(x[n]) for n in ("q", "k", "v", "log_a", "S0")]
    o, S = bo.gated_recurrence(*a)
    ab = [None if y is None else np.abs(y) for y in a]
    ab[3] = a[3]
    ao, aS = bo.gated_recurrence(*ab)
    return o, S, ao, aS


def _meets(name, got, ref, size, factor):
    got = _np(got)
    assert got.shape == ref.shape, name
    tol = factor * U * np.maximum(size, 1e-6 * np.mean(size))
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d off, worst %g times the tolerance" % (
        name, bad.sum(), np.nanmax(np.abs(got - ref)[bad] / np.maximum(tol[bad], 1e-300)))


def _factor(L, dk, dv):
    return dk + dv + 80 + 8 * (-(-L // 64))


DIMS = [(16, 16), (16, 128), (32, 32), (64, 64), (128, 16), (64, 32), (32, 64), (128, 64), (128, 128)]
LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 130, 321]


def _check_forward(x, **kw):
    B, H, L, dk = x["q"].shape
    o, S = fw.gated_fwd_chunk(x["q"], x["k"], x["v"], x["log_a"], S0=x["S0"], return_state=True, **kw)
    ro, rS, ao, aS = _forward_ref(x)
    f = _factor(L, dk, x["v"].shape[-1])
    _meets("o", o, ro, ao, f)
    _meets("S", S, rS, aS, f)
    return o, S


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("L", LENGTHS)
def test_forward(dtype, dk, dv, L):
    gate = ["mixed", "strong", "resets", "none"][(L + dk + dv) % 4]
    _check_forward(_inputs(L, 2, 3, L, dk, dv, dtype, gate=gate, start=L % 2 == 1))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gate", ["mixed", "strong", "resets", "none"])
@pytest.mark.parametrize("start", [False, True])
def test_forward_gates(dtype, gate, start):
    _check_forward(_inputs(7, 1, 2, 200, 64, 64, dtype, gate=gate, start=start))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv,L", [(64, 64, 2049), (128, 128, 1100), (16, 32, 4000), (32, 128, 777)])
def test_forward_in_segments(dtype, dk, dv, L):
    """Long sequences of few heads: the call cut into segments and the one in order
    both meet the recurrence; each is the same bits every time."""
    x = _inputs(8, 1, 2, L, dk, dv, dtype, gate="resets")
    need = fw.load_library().falcon_gated_fwd_workspace_bytes(1, 2, L, dk, dv, int(dtype == torch.float32))
    assert need > 0
    o, S = _check_forward(x)
    o2, S2 = _check_forward(x, workspace=torch.empty(need + 100, device="cuda", dtype=torch.uint8))
    assert torch.equal(o, o2) and torch.equal(S, S2)
    o3, S3 = _check_forward(x, workspace=None)
    o4, S4 = _check_forward(x, workspace=torch.empty(max(need - 16, 0), device="cuda", dtype=torch.uint8))
    assert torch.equal(o3, o4) and torch.equal(S3, S4)
    # the state written over the one that the call starts from
    S5 = x["S0"].clone()
    o5 = fw.gated_fwd_chunk(x["q"], x["k"], x["v"], x["log_a"], S0=S5, S_out=S5)
    assert torch.equal(o5, o) and torch.equal(S5, S)


def test_resumed_sequence_and_single_tokens():
    """A sequence in pieces, the last ones single tokens, against one call's oracle."""
    L, cuts = 150, [0, 1, 65, 100, 147, 148, 149, 150]
    x = _inputs(9, 2, 2, L, 64, 64, torch.bfloat16)
    S, parts = x["S0"].clone(), []
    for a, b in zip(cuts, cuts[1:]):
        q, k, v = (x[n][:, :, a:b].contiguous() for n in ("q", "k", "v"))
        la = x["log_a"][:, :, a:b].contiguous()
        if b - a == 1:
            parts.append(fw.gated_decode_step(S, q[:, :, 0].contiguous(), k[:, :, 0].contiguous(),
                                              v[:, :, 0].contiguous(), la[:, :, 0].contiguous())[:, :, None])
        else:
            parts.append(fw.gated_fwd_chunk(q, k, v, la, S0=S, S_out=S))
    ro, rS, ao, aS = _forward_ref(x)
    _meets("o", torch.cat(parts, 2), ro, ao, _factor(L, 64, 64) + 8 * len(cuts))
    _meets("S", S, rS, aS, _factor(L, 64, 64) + 8 * len(cuts))


def test_many_chains_and_rows_behind():
    """More chains than segments are cut for; memory behind and before o untouched."""
    x = _inputs(10, 70, 12, 70, 16, 16, torch.bfloat16)
    buf = torch.full((70 * 12 * 70 * 16 + 512,), 7.0, device="cuda")
    out = buf[256:-256].view(70, 12, 70, 16)
    o, _ = _check_forward(x, out=out)
    assert bool((buf[:256] == 7).all()) and bool((buf[-256:] == 7).all())


def _backward(x, seed, *, end=True, **kw):
    r = np.random.default_rng(seed)
    B, H, L, dk = x["q"].shape
    dv = x["v"].shape[-1]
    dO = _up(r.standard_normal((B, H, L, dv)))
    dS = _up(0.3 * r.standard_normal((B, H, dv, dk))) if end else None
    return dO, dS, fw.gated_bwd_chunk(x["q"], x["k"], x["v"], x["log_a"], dO, S0=x["S0"], dS_L=dS, **kw)


def _check_backward(x, seed, **kw):
    """dlog_a's terms: r and c are dot products of an output with an input (d more terms),
    and a segment's sums add up to 1024 of each: an error of every r and c before it,
    f u of each one's own size, beside X's.  All bounds on absolute sums."""
    dO, dS, got = _backward(x, seed, **kw)
    B, H, L, dk = x["q"].shape
    dv = x["v"].shape[-1]
    a = [_np(x[n]) for n in ("q", "k", "v", "log_a")]
    ref = bo.gated_backward(*a, _np(dO), _np(x["S0"]), _np(dS))
    ab = [None if y is None else np.abs(y) for y in a]
    ab[3] = a[3]
    size = bo.gated_backward(*ab, np.abs(_np(dO)), None if x["S0"] is None else np.abs(_np(x["S0"])),
                             None if dS is None else np.abs(_np(dS)))
    f = _factor(L, dk, dv) + max(dk, dv)
    for n in ("dq", "dk", "dv"):
        _meets(n, got[n], ref[n], size[n], f)
    assert ("dS0" in got) == (x["S0"] is not None) and ("dlog_a" in got) == (x["log_a"] is not None)
    if "dS0" in got:
        _meets("dS0", got["dS0"], ref["dS0"], size["dS0"], f)
    if "dlog_a" in got:
        # sizes of r and c over the segment (1024 tokens at most), the borders' own beside
        rc = np.sum(np.abs(a[0]) * size["dq"], -1) + np.sum(np.abs(a[1]) * size["dk"], -1)
        behind = np.cumsum(rc[..., ::-1], -1)[..., ::-1]
        behind[..., :-1024] -= behind[..., 1024:]
        top = np.max(size["dlog_a"], axis=-1, keepdims=True)
        _meets("dlog_a", got["dlog_a"], ref["dlog_a"], behind + top, f)
        # and as a whole: the errors of a sum's terms do not all point one way
        err = np.linalg.norm(_np(got["dlog_a"]) - ref["dlog_a"])
        assert err <= 2e-5 * np.linalg.norm(ref["dlog_a"]) + 1e-6
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("L", LENGTHS)
def test_backward(dtype, dk, dv, L):
    gate = ["mixed", "strong", "resets", "none"][(L + dk + dv) % 4]
    _check_backward(_inputs(L, 2, 3, L, dk, dv, dtype, gate=gate, start=L % 2 == 1), 20, end=L % 3 != 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gate", ["mixed", "strong", "resets", "none"])
@pytest.mark.parametrize("start,end", [(False, False), (True, False), (False, True), (True, True)])
def test_backward_gates(dtype, gate, start, end):
    _check_backward(_inputs(21, 1, 2, 200, 64, 64, dtype, gate=gate, start=start), 22, end=end)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv,L", [(64, 64, 2049), (128, 128, 1100), (16, 32, 4000), (32, 128, 777)])
def test_backward_in_segments(dtype, dk, dv, L):
    x = _inputs(23, 1, 2, L, dk, dv, dtype, gate="mixed")
    got = _check_backward(x, 24)
    again = _backward(x, 24)[2]
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("L", [900, 1100])
def test_backward_of_many_chains(L):
    """Segments of 1024 tokens at most, whatever the number of chains: one and two."""
    _check_backward(_inputs(25, 30, 40, L, 16, 16, torch.bfloat16, gate="resets"), 26)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64), (torch.float32, 128)])
def test_captured_with_large_lds(dtype, d):
    """Kernels with more than 64 KB of LDS, captured and replayed on other inputs."""
    xs = [_inputs(40 + i, 1, 2, 600, d, d, dtype) for i in range(2)]
    dO = _up(np.random.default_rng(42).standard_normal((1, 2, 600, d)))

    def run(x):
        o, S = fw.gated_fwd_chunk(x["q"], x["k"], x["v"], x["log_a"], S0=x["S0"], return_state=True)
        g = fw.gated_bwd_chunk(x["q"], x["k"], x["v"], x["log_a"], dO, S0=x["S0"], dS_L=S)
        return [o, S] + [g[n] for n in sorted(g)]
    want = [[t.clone() for t in run(x)] for x in xs]
    bound = {n: t.clone() for n, t in xs[0].items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(bound)
    for rep in (0, 1, 0, 1):
        for n, t in bound.items():
            t.copy_(xs[rep][n])
        graph.replay()
        run(xs[rep])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[rep])), rep


def test_log_decays_of_any_alignment():
    """A step's log decays as a slice of all steps' (4-byte aligned), three heads."""
    x = _inputs(46, 1, 3, 70, 32, 16, torch.bfloat16)
    buf = torch.zeros(3 * 70 + 8, device="cuda")
    dO = _up(np.random.default_rng(47).standard_normal((1, 3, 70, 16)))
    run = lambda la: [fw.gated_fwd_chunk(x["q"], x["k"], x["v"], la, S0=x["S0"])] + list(  # noqa: E731
        fw.gated_bwd_chunk(x["q"], x["k"], x["v"], la, dO).values())
    want = run(x["log_a"])
    for at in (1, 2, 3):
        la = buf[at:at + 210].view(1, 3, 70)
        la.copy_(x["log_a"])
        assert all(torch.equal(a, b) for a, b in zip(run(la), want))
    steps = -torch.rand(4, 1, 3, device="cuda")
    for t in range(4):
        S, S2 = x["S0"].clone(), x["S0"].clone()
        one = [x[n][:, :, t].contiguous() for n in ("q", "k", "v")]
        o = fw.gated_decode_step(S, *one, steps[t])
        assert torch.equal(o, fw.gated_decode_step(S2, *one, steps[t].clone())) and torch.equal(S, S2)


def test_growing_state():
    """log_a > 0: gates above one, the state grows by e^(0.05 L)."""
    x = _inputs(43, 1, 2, 200, 32, 64, torch.bfloat16)
    x["log_a"] = x["log_a"].abs() * 0.5
    x["log_a"][..., ::7] *= -1
    _check_forward(x)
    _check_backward(x, 44)


def test_offsets_beyond_32_bits():
    """One chain of nine million tokens of 128 columns (o is 4.6 GB): the last 100 tokens,
    behind a reset, are a sequence of their own, and their gradients too."""
    L, n, d = 9_000_011, 100, 128
    tail = _inputs(45, 1, 1, n, d, d, torch.bfloat16, start=False)
    tail["log_a"][..., 0] = -float("inf")
    x = {m: torch.full((1, 1, L, d), 0.01, device="cuda", dtype=torch.bfloat16) for m in ("q", "k", "v")}
    x["log_a"] = torch.full((1, 1, L), -0.1, device="cuda")
    for m, t in x.items():
        t[:, :, -n:] = tail[m]
    dO = torch.zeros((1, 1, L, d), device="cuda")
    dO[:, :, -n:] = 1.0
    o, S = fw.gated_fwd_chunk(x["q"], x["k"], x["v"], x["log_a"], return_state=True)
    ro, rS, ao, aS = _forward_ref(tail)
    _meets("o", o[:, :, -n:], ro, ao, _factor(n + 64, d, d))
    _meets("S", S, rS, aS, _factor(n + 64, d, d))
    del o
    g = fw.gated_bwd_chunk(x["q"], x["k"], x["v"], x["log_a"], dO)
    a = [_np(tail[m]) for m in ("q", "k", "v", "log_a")]
    ones = np.ones((1, 1, n, d))
    ref = bo.gated_backward(*a, ones)
    size = bo.gated_backward(*[np.abs(y) for y in a[:3]], a[3], ones)
    for m in ("dq", "dk", "dv"):
        _meets(m, g[m][:, :, -n:], ref[m], size[m], _factor(n + 64, d, d) + d)
        assert not g[m][:, :, :-n].any()                # nothing passes the reset
    assert not g["dlog_a"][:, :, :-n + 1].any()


def test_backward_against_differences():
    """Along random directions, central differences of the fp64 recurrence: their own
    error is about 1e-8 of values of order one, the kernels' 1e-5 of the absolute sum."""
    x = _inputs(27, 1, 2, 100, 32, 64, torch.float32)
    dO, dS, d = _backward(x, 28)
    base = [_np(x[n]) for n in ("q", "k", "v", "log_a", "S0")]
    r = np.random.default_rng(29)
    for i, n in enumerate(("dq", "dk", "dv", "dlog_a", "dS0")):
        u = r.standard_normal(base[i].shape)

        def f(h):
            y = list(base)
            y[i] = y[i] + h * u
            o, S = bo.gated_recurrence(*y)
            return np.sum(o * _np(dO)) + np.sum(S * _np(dS))
        want, have = (f(1e-5) - f(-1e-5)) / 2e-5, np.sum(_np(d[n]) * u)
        assert abs(want - have) <= 1e-6 + 1e-5 * np.sum(np.abs(_np(d[n]) * u)), n


@pytest.mark.parametrize("seed", range(60))
def test_random_configurations(seed):
    """Sizes, types, gates and starts drawn at random: every block size, cut and whole
    sequences, forward, gradients and a decode step behind the sequence."""
    r = np.random.default_rng(1000 + seed)
    dk, dv = (int(r.choice([16, 32, 64, 128])) for _ in range(2))
    L = int(np.exp(r.uniform(0, np.log(1500))))
    B, H = int(r.integers(1, 4)), int(r.integers(1, 7))
    if L * B * H * max(dk, dv) > 400_000:
        B, H = 1, min(H, 2)
    dtype = TYPES[int(r.integers(2))]
    x = _inputs(seed, B, H, L, dk, dv, dtype, gate=str(r.choice(["mixed", "strong", "resets", "none"])),
                start=bool(r.integers(2)))
    _, S = _check_forward(x)
    _check_backward(x, seed + 500, end=bool(r.integers(2)))
    q, k, v = (x[n][:, :, -1].contiguous() for n in ("q", "k", "v"))
    la = None if x["log_a"] is None else x["log_a"][:, :, -1].contiguous()
    one = fw.gated_fwd_chunk(*(t[:, :, None] for t in (q, k, v)), None if la is None else la[:, :, None],
                             S0=S, return_state=True)
    o = fw.gated_decode_step(S, q, k, v, la)
    for a, b in ((o, one[0][:, :, 0]), (S, one[1])):
        assert float((a - b).norm()) <= 1e-6 * float(b.norm()) + 1e-30
