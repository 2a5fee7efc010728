"""The gated delta rule's chunk forward, gradients and decode step against the fp64 rule;
bounds in delta_util."""
import numpy as np
import pytest

import delta_util as du
from oracle import delta_oracle as do

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import weight_recurrent_memory_amd as fw  # noqa: E402
from weight_recurrent_memory_amd import block_binding  # noqa: E402

TYPES = [torch.bfloat16, torch.float32]
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    block_binding.load_library()


def _forward(x, **kw):
    return fw.gated_delta_fwd_chunk(x["q"], x["k"], x["v"], x["beta"], x["log_a"], S0=x["S0"], **kw)


def _backward(x, dS_L=True, **kw):
    return fw.gated_delta_bwd_chunk(x["q"], x["k"], x["v"], x["beta"], x["log_a"], x["dO"], S0=x["S0"],
                                    dS_L=x["dS_L"] if dS_L else None, **kw)


def _check_forward(x, bound=du.FORWARD):
    o, S = _forward(x, return_state=True)
    ro, rS, _, _ = du.recurrence(torch, x)
    assert du.off(o, ro) <= bound and du.off(S, rS) <= bound, (du.off(o, ro), du.off(S, rS))
    return o, S


def _check_backward(x, dS_L=True, bound=du.GRADIENT):
    got, ref = _backward(x, dS_L), du.gradients(torch, x, dS_L)
    assert set(got) == {"dq", "dk", "dv", "dbeta"} | ({"dlog_a"} if x["log_a"] is not None else set()) \
        | ({"dS0"} if x["S0"] is not None else set())
    for n in got:
        if n in ("dlog_a", "dbeta"):
            # differences: dbeta = du . v - y . k, dlog_a a running sum of q . dq - v . dv over up
            # to 64 tokens, whose errors add up as a root of 64 squares at most
            terms = {"dlog_a": 8 * (du.norm((x["q"].double() * ref["dq"]).sum(-1))
                                    + du.norm((x["v"].double() * ref["dv"]).sum(-1))),
                     "dbeta": du.norm((x["v"].double() * ref["dv"]).sum(-1) / x["beta"].double().clamp(min=0.1))}[n]
            assert du.norm(got[n].double() - ref[n]) <= bound * (du.norm(ref[n]) + terms), n
        else:
            assert du.norm(got[n].double() - ref[n]) <= bound * max(du.norm(ref[n]), 1e-12), (n, du.off(got[n], ref[n]))
    return got


DIMS = [(16, 16), (16, 128), (32, 32), (64, 64), (128, 16), (64, 32), (32, 64), (128, 64), (128, 128)]
LENGTHS = [1, 2, 15, 17, 63, 64, 65, 130]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("L", LENGTHS)
def test_forward(dtype, dk, dv, L):
    gate = ["mixed", "strong", "resets", "none"][(L + dk + dv) % 4]
    _check_forward(du.inputs(torch, L, 2, 3, L, dk, dv, dtype, gate=gate, start=L % 2 == 1))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("L", [1, 17, 64, 65, 130])
def test_backward(dtype, dk, dv, L):
    gate = ["mixed", "strong", "resets", "none"][(L + dk + dv) % 4]
    _check_backward(du.inputs(torch, L, 1, 3, L, dk, dv, dtype, gate=gate, start=L % 2 == 1), dS_L=L % 2 == 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gate", ["mixed", "strong", "resets", "none"])
@pytest.mark.parametrize("beta", ["mixed", "one", "zero", "two"])
def test_gates_and_strengths(dtype, gate, beta):
    x = du.inputs(torch, 7, 1, 2, 150, 64, 64, dtype, gate=gate, beta=beta)
    _check_forward(x)
    _check_backward(x)


@pytest.mark.parametrize("beta", ["mixed", "one"])
def test_repeated_keys(beta):
    """Keys repeated 40 times: T's entries cancel.  (bf16 keys are unit to 2^-8: a step of
    beta |k|^2 up to 1.01.)"""
    for dtype in TYPES:
        x = du.inputs(torch, 8, 2, 2, 200, 32, 32, dtype, beta=beta, keys="repeated", gate="none")
        _check_forward(x)
        _check_backward(x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv,L", [(64, 64, 2049), (128, 128, 1100), (16, 32, 4000), (32, 128, 1500), (16, 16, 1030)])
def test_long_sequences_of_few_heads(dtype, dk, dv, L):
    x = du.inputs(torch, 9, 1, 2, L, dk, dv, dtype, gate="resets")
    o, S = _check_forward(x)
    need = block_binding.load_library().falcon_gated_delta_fwd_workspace_bytes(1, 2, L, dk, dv, int(dtype == torch.float32))
    o2, S2 = _forward(x, return_state=True, workspace=torch.empty(need, device="cuda", dtype=torch.uint8))
    assert torch.equal(o, o2) and torch.equal(S, S2)
    d, d2 = _check_backward(x), _backward(x)
    assert all(torch.equal(d[n], d2[n]) for n in d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("beta", ["mixed", "zero"])
@pytest.mark.parametrize("H,dk,dv,L", [(1, 128, 128, 576), (1, 128, 128, 640), (1, 128, 64, 703), (20, 128, 128, 1100),
                                       (3, 64, 64, 640), (27, 64, 64, 1000), (5, 32, 16, 641), (3, 16, 64, 1999)])
def test_what_segments_hand_on(dtype, beta, H, dk, dv, L):
    """No decay, half of the keys without a step: a segment's matrix is far from zero, and the
    start's share reaches the last segments.  (A join adds one product a segment, up to 8u each of
    what the decreasing starts hold; the roundings point either way, and the bounds hold twice the
    rest.)"""
    x = du.inputs(torch, 23, 1, H, L, dk, dv, dtype, gate="none", beta=beta)
    _check_forward(x)
    _check_backward(x)


@pytest.mark.parametrize("L", [100, 1500])
def test_state_in_place_and_given_outputs(L):
    x = du.inputs(torch, 10, 1, 2, L, 32, 32, torch.bfloat16)
    o, S = _forward(x, return_state=True)
    kept, out = x["S0"].clone(), torch.full((1, 2, L, 32), NAN, device="cuda")
    o2 = fw.gated_delta_fwd_chunk(x["q"], x["k"], x["v"], x["beta"], x["log_a"], S0=kept, S_out=kept, out=out)
    assert o2 is out and torch.equal(o, out) and torch.equal(S, kept)


@pytest.mark.parametrize("start,end", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("L", [70, 1500])
def test_gradients_of_either_end(start, end, L):
    _check_backward(du.inputs(torch, 21, 1, 2, L, 32, 64, torch.bfloat16, start=start), dS_L=end)


def test_gates_of_any_alignment():
    """beta and log_a as views that start at an odd element."""
    x = du.inputs(torch, 22, 1, 3, 130, 32, 32, torch.bfloat16)
    want, wantb = _forward(x), _backward(x)
    for n in ("beta", "log_a"):
        room = torch.empty(x[n].numel() + 3, device="cuda")
        room[3:].copy_(x[n].flatten())
        x[n] = room[3:].view(1, 3, 130)
        assert x[n].data_ptr() % 16
    got = _backward(x)
    assert torch.equal(_forward(x), want) and all(torch.equal(got[n], wantb[n]) for n in got)


def test_rows_behind_the_outputs_stay():
    x = du.inputs(torch, 11, 1, 3, 70, 16, 16, torch.bfloat16)
    room = torch.full((3 * 70 * 16 + 64,), 7.0, device="cuda")
    fw.gated_delta_fwd_chunk(x["q"], x["k"], x["v"], x["beta"], x["log_a"], out=room[:-64].view(1, 3, 70, 16))
    assert torch.all(room[-64:] == 7.0) and torch.all(torch.isfinite(room))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", DIMS)
def test_decode_is_the_sequence_token_by_token(dtype, dk, dv):
    L = 9
    x = du.inputs(torch, 12, 3, 5, L, dk, dv, dtype, gate="resets")
    ro, rS, _, _ = du.recurrence(torch, x)
    S = x["S0"].clone()
    for t in range(L):
        o = fw.gated_delta_decode_step(S, *(x[n][:, :, t].contiguous() for n in ("q", "k", "v", "beta", "log_a")))
        # a step: one product of dk terms, its rounding and the state's
        assert du.off(o, ro[:, :, t]) <= du.FORWARD
    assert du.off(S, rS) <= du.FORWARD


def test_decode_without_decay():
    x = du.inputs(torch, 13, 2, 2, 1, 64, 64, torch.bfloat16, gate="none")
    S = x["S0"].clone()
    o = fw.gated_delta_decode_step(S, *(x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "beta")))
    ro, rS, _, _ = du.recurrence(torch, x)
    assert du.off(o, ro[:, :, 0]) <= du.FORWARD and du.off(S, rS) <= du.FORWARD


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [70, 1500])
@pytest.mark.parametrize("which", ["v", "k", "q", "beta", "log_a"])
@pytest.mark.parametrize("value", [NAN, INF])
def test_what_is_not_finite_stays_where_it_is_read(dtype, L, which, value):
    """A NaN or an infinity at token t of one head: o before it and the other heads' as
    without it; with one in v, so are the other value rows."""
    if which == "log_a" and value == INF:
        value = NAN
    x = du.inputs(torch, 14, 1, 3, L, 32, 32, dtype)
    o, S = _forward(x, return_state=True)
    t = L - 33
    y = dict(x, **{which: x[which].clone()})
    if which in ("q", "k", "v"):
        y[which][0, 1, t, 5] = value
    else:
        y[which][0, 1, t] = value
    o2, S2 = _forward(y, return_state=True)
    near = lambda a, b: du.norm(a.double() - b.double()) <= 2 * du.FORWARD * du.norm(b)  # noqa: E731
    assert near(o2[:, ::2], o[:, ::2]) and near(S2[:, ::2], S[:, ::2])
    assert near(o2[:, 1, :t], o[:, 1, :t])
    if which == "q":
        assert torch.equal(S2, S) and near(o2[:, 1, t + 1:], o[:, 1, t + 1:])
        assert not torch.isfinite(o2[0, 1, t]).any()
        return
    rows = [5] if which == "v" else list(range(32))
    rest = [i for i in range(32) if i not in rows]
    assert not torch.isfinite(o2[0, 1, t, rows]).any() and not torch.isfinite(S2[0, 1, rows]).all()
    if rest:
        assert near(o2[0, 1][:, rest], o[0, 1][:, rest]) and near(S2[0, 1, rest], S[0, 1, rest])


def test_padding_may_hold_anything():
    """A batch of unequal lengths: what lies behind a sequence leaves its outputs alone."""
    x = du.inputs(torch, 15, 2, 2, 100, 64, 64, torch.bfloat16)
    o = _forward(x)
    y = {n: t.clone() if t is not None else None for n, t in x.items()}
    for n in ("q", "k", "v", "beta", "log_a"):
        y[n][1, :, 60:] = NAN
    o2 = _forward(y)
    assert du.off(o2[0], o[0].double()) <= 2 * du.FORWARD
    assert du.off(o2[1, :, :60], o[1, :, :60].double()) <= 2 * du.FORWARD


def test_gradients_are_the_formulas_and_differences():
    """Against the numpy form, and a difference of the library's own forward: a step h gives
    2^-24 |loss| / h of rounding and h^2 of curvature."""
    x = du.inputs(torch, 16, 1, 2, 80, 16, 16, torch.float32, gate="mixed")
    n = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    ref = do.delta_backward(*(n(x[m]) for m in ("q", "k", "v", "beta", "log_a", "dO", "S0", "dS_L")))
    got = _backward(x)
    for m in ref:
        assert np.linalg.norm(n(got[m]) - ref[m]) <= 8 * du.GRADIENT * np.linalg.norm(ref[m]), m

    def loss(y):
        o, S = _forward(y, return_state=True)
        return float((o.double() * x["dO"]).sum() + (S.double() * x["dS_L"]).sum())
    g = torch.Generator(device="cuda").manual_seed(1)
    for m in ("q", "k", "v", "beta", "log_a", "S0"):
        u = torch.randn(x[m].shape, generator=g, device="cuda") * (0.1 if m in ("beta", "log_a") else 1.0)
        h = 2.0 ** -10
        d = (loss(dict(x, **{m: x[m] + h * u})) - loss(dict(x, **{m: x[m] - h * u}))) / (2 * h)
        want = float((got["d" + m].double() * u).sum())
        size = float((got["d" + m].double().abs() * u.abs()).sum())
        # |loss| is below 200 here; rounding of two forwards, and h^2 of third derivatives
        assert abs(d - want) <= 2 * 200 * du.FORWARD / h + 100 * h * h * max(size, 1.0), (m, d, want)


def test_captured_with_an_eager_call_between():
    """Forward, gradients and a decode step in one graph, replayed on new inputs."""
    x = du.inputs(torch, 17, 2, 3, 150, 64, 32, torch.bfloat16, gate="resets")
    one = du.inputs(torch, 18, 2, 3, 1, 64, 32, torch.bfloat16)
    tok = {n: one[n][:, :, 0].contiguous() for n in ("q", "k", "v", "beta", "log_a")}
    S = one["S0"].clone()

    def step():
        o, S_L = _forward(x, return_state=True)
        return [o, S_L, fw.gated_delta_decode_step(S, **tok), *_backward(x).values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for seed in range(3):
        new, S_new = du.inputs(torch, 30 + seed, 2, 3, 150, 64, 32, torch.bfloat16, gate="resets"), torch.randn_like(S)
        for n, t in x.items():
            t.copy_(new[n])
        S.copy_(S_new)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        S.copy_(S_new)
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_other_streams_and_two_calls_at_once():
    x, y = (du.inputs(torch, 19 + i, 2, 4, 300, 64, 64, torch.bfloat16) for i in range(2))
    want = [_forward(x), _forward(y)]
    wantb = [_backward(x), _backward(y)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [_forward(x, stream=s[0]), _forward(y, stream=s[1].cuda_stream)]
    gotb = [_backward(x, stream=s[0]), _backward(y, stream=s[1])]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a[n], b[n]) for a, b in zip(gotb, wantb) for n in a)


def test_offsets_beyond_32_bits():
    """2^32 bytes of o and more: the last head's outputs as those of a call of its own."""
    H, L = 66, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(20)
    q, k, v = (torch.randn((1, H, L, 16), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    for t in (q, k):
        t.mul_(0.25)                     # about unit rows
    beta = torch.full((1, H, L), 0.3, device="cuda")
    log_a = torch.full((1, H, L), -0.01, device="cuda")
    o, S = fw.gated_delta_fwd_chunk(q, k, v, beta, log_a, return_state=True)
    last = lambda t: t[:, -1:].contiguous()  # noqa: E731
    o1, S1 = fw.gated_delta_fwd_chunk(last(q), last(k), last(v), last(beta), last(log_a), return_state=True)
    assert du.off(o[:, -1:], o1.double()) <= 2 * du.FORWARD and du.off(S[:, -1:], S1.double()) <= 2 * du.FORWARD
