"""The norms and the recurrences together, as a block between two projections runs them:
forward and backward, captured in a graph, on another stream, then token by token."""
import numpy as np
import pytest

from oracle import block_oracle as bo
from oracle import falcon_oracle as fo

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import weight_recurrent_memory_amd as fw  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fw.load_library()


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, ref, rel):
    """2-norms: an error of one part in `rel` of the whole."""
    assert np.linalg.norm(_np(got) - ref) <= rel * np.linalg.norm(ref)


B, L, H, DK, DV = 2, 150, 3, 32, 64
WIDTH = H * (2 * DK + 2 * DV)


def _batch(seed, dtype, b=B, l=L):
    """One fused projection's rows (q, k, v, gate), log decays, weight, residual, dy."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    p = rn(b, l, WIDTH).to(dtype)
    return dict(p=p, log_a=torch.nn.functional.logsigmoid(rn(b, H, l) + 3), w=1 + 0.1 * rn(DV),
                res=rn(b, l, H, DV).to(dtype), dy=rn(b, l, H, DV).to(dtype), S0=0.2 * rn(b, H, DV, DK))


def _views(p):
    b, l, _ = p.shape
    at, out = 0, []
    for d in (DK, DK, DV, DV):
        out.append(p[..., at:at + H * d].view(b, l, H, d))
        at += H * d
    return out


def _forward(x, update):
    q_in, k_in, v_in, gate = _views(x["p"])
    q, k, v = fw.norm_in(q_in, k_in, v_in)
    o = update(q, k, v)
    return q, k, v, o, fw.norm_out(o, x["w"], gate, residual=x["res"], scale=0.5)


def _backward(x, kept, gradients):
    q_in, k_in, _, gate = _views(x["p"])
    q, k, v, o, _ = kept
    dp = torch.empty_like(x["p"])
    dq_in, dk_in, dv_in, dgate = _views(dp)
    n = fw.norm_out_bwd(o, x["w"], x["dy"], gate, scale=0.5, dgate=dgate)
    d = gradients(q, k, v, n["dO"])
    fw.norm_in_bwd(q_in, k_in, d["dq"], d["dk"], d["dv"], out=(dq_in, dk_in, dv_in))
    return dp, n["dweight"], d


def _gated(x):
    return (lambda q, k, v: fw.gated_fwd_chunk(q, k, v, x["log_a"], S0=x["S0"]),
            lambda q, k, v, dO: fw.gated_bwd_chunk(q, k, v, x["log_a"], dO, S0=x["S0"]))


def _falcon(x):
    kw = dict(variant=fw.FALCON_1, beta=0.5, lam=0.05, eps=1e-6)
    return (lambda q, k, v: fw.fwd_recurrent(q, k, v, **kw),
            lambda q, k, v, dO: fw.bwd_chunk(q, k, v, dO, **kw))


def _reference(x, update, gradients):
    """The same block in fp64, numpy."""
    hf = lambda t: np.swapaxes(t, 1, 2)  # noqa: E731
    q_in, k_in, v_in, gate = (_np(t) for t in _views(x["p"]))
    q, k, v = bo.unit_rows(hf(q_in), 1e-6), bo.unit_rows(hf(k_in), 1e-6), hf(v_in)
    o = update(q, k, v)
    y = bo.norm_out(o, _np(x["w"]), gate, "silu", _np(x["res"]), 0.5, 1e-6)
    n = bo.norm_out_backward(o, _np(x["w"]), _np(x["dy"]), gate, "silu", 0.5, 1e-6)
    d = gradients(q, k, v, n["dO"])
    parts = [bo.unit_rows_backward(q_in, hf(d["dq"]), 1e-6), bo.unit_rows_backward(k_in, hf(d["dk"]), 1e-6),
             hf(d["dv"]), n["dgate"]]
    b, l = q_in.shape[:2]
    return y, np.concatenate([t.reshape(b, l, -1) for t in parts], -1), n["dweight"], d


def test_block_with_the_gated_recurrence():
    """float32 from end to end: four stages of sums of up to 150 terms, each good to about
    1e-6 of its result, none amplifying an error by more than the norms' condition (rows
    of 64 independent entries: a few), so 1e-4 holds with an order of magnitude to spare."""
    x = _batch(1, torch.float32)
    up, grad = _gated(x)
    kept = _forward(x, up)
    dp, dw, d = _backward(x, kept, grad)
    la, S0 = _np(x["log_a"]), _np(x["S0"])
    y, rp, rw, rd = _reference(x, lambda q, k, v: bo.gated_recurrence(q, k, v, la, S0)[0],
                               lambda q, k, v, dO: bo.gated_backward(q, k, v, la, dO, S0))
    for got, ref in ((kept[-1], y), (dp, rp), (dw, rw), (d["dlog_a"], rd["dlog_a"]), (d["dS0"], rd["dS0"])):
        _close(got, ref, 1e-4)


def test_block_with_a_falcon_rule():
    """The norms around the library's own update (float32: the recurrent form and its
    gradients, whose own gates are 1e-4 relative to the largest entry)."""
    x = _batch(2, torch.float32)
    up, grad = _falcon(x)
    kept = _forward(x, up)
    dp, dw, _ = _backward(x, kept, grad)
    kw = dict(beta=0.5, lam=0.05, eps=1e-6)
    y, rp, rw, _ = _reference(x, lambda q, k, v: fo.falcon_recurrence(0, q, k, v, **kw)[0],
                              lambda q, k, v, dO: fo.falcon_backward(0, q, k, v, dO, **kw))
    for got, ref in ((kept[-1], y), (dp, rp), (dw, rw)):
        _close(got, ref, 5e-4)


def test_block_captured_and_replayed():
    """Forward and backward in one graph, new inputs copied in between replays, an eager
    run of the same tensors alive beside it: the eager results' bits every time."""
    x = _batch(3, torch.bfloat16, l=700)
    other = _batch(4, torch.bfloat16, l=700)
    run = lambda z: (lambda kept: kept + _backward(z, kept, _gated(z)[1])[:2])(_forward(z, _gated(z)[0]))  # noqa: E731
    eager = [t.clone() for t in run(x)]
    live = run(x)
    want = {id(x): eager, id(other): [t.clone() for t in run(other)]}
    bound = {n: t.clone() for n, t in x.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(bound)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(bound)
    for rep, z in enumerate((x, other, x, other)):
        for n, t in bound.items():
            t.copy_(z[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[id(z)])), rep
        assert all(torch.equal(a, b) for a, b in zip(live, eager))
        run(x)                                     # eager work between replays
        torch.cuda.synchronize()


def test_another_stream():
    """stream=: the call and what it allocates belong to that stream."""
    x = _batch(5, torch.bfloat16, l=700)
    q_in, k_in, v_in, gate = _views(x["p"])
    up, _ = _gated(x)
    want = _forward(x, up)
    grads = fw.gated_bwd_chunk(*want[:3], x["log_a"], want[3], S0=x["S0"])
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        q, k, v = fw.norm_in(q_in, k_in, v_in, stream=stream)
        o = fw.gated_fwd_chunk(q, k, v, x["log_a"], S0=x["S0"], stream=stream)
        y = fw.norm_out(o, x["w"], gate, residual=x["res"], scale=0.5, stream=stream)
        d = fw.gated_bwd_chunk(q, k, v, x["log_a"], o, S0=x["S0"], stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip((q, k, v, o, y), want))
        assert all(torch.equal(d[n], grads[n]) for n in grads)


def test_default_stream_by_its_handle_and_empty_calls():
    x = _batch(9, torch.bfloat16, l=20)
    q_in, k_in, v_in, _ = _views(x["p"])
    torch.cuda.synchronize()
    q, k, v = fw.norm_in(q_in, k_in, v_in, stream=0)
    torch.cuda.synchronize()
    want = fw.norm_in(q_in, k_in, v_in)
    assert all(torch.equal(a, b) for a, b in zip((q, k, v), want))
    # no tokens, no sequences: refused as by the other entry points
    none = q[:, :, :0].contiguous()
    for call in (lambda: fw.gated_fwd_chunk(none, none, v[:, :, :0].contiguous()),
                 lambda: fw.gated_fwd_chunk(q[:0], k[:0], v[:0]),
                 lambda: fw.norm_in(q_in[:, :0], k_in[:, :0]),
                 lambda: fw.norm_out(q[:, :, :0].float(), torch.ones(DK, device="cuda")),
                 lambda: fw.gated_decode_step(x["S0"][:0], q[:0, :, 0], k[:0, :, 0], v[:0, :, 0])):
        with pytest.raises((fw.FalconError, ValueError)):
            call()


def test_two_calls_at_once():
    """Two streams, two batches, no workspace in common."""
    xs = [_batch(6 + i, torch.bfloat16, l=900) for i in range(2)]
    want = [[t.clone() for t in _forward(x, _gated(x)[0])] for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for s, x in zip(streams, xs):
        with torch.cuda.stream(s):
            got.append([_forward(x, _gated(x)[0]) for _ in range(3)])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for run in g for a, b in zip(run, w))


def test_prefill_then_single_tokens():
    """A prompt in one call, then tokens one by one through the norms and the decode
    step, against the whole sequence's fp64 recurrence from the same unit rows."""
    n, l = 3, 40
    x = _batch(8, torch.bfloat16, b=n, l=l)
    q_in, k_in, v_in, gate = _views(x["p"])
    cut = 30
    part = lambda t, a, b: t[:, a:b]  # noqa: E731
    q, k, v = fw.norm_in(*(part(t, 0, cut).contiguous() for t in (q_in, k_in, v_in)))
    S = x["S0"].clone()
    la = x["log_a"]
    o, S = fw.gated_fwd_chunk(q, k, v, la[:, :, :cut].contiguous(), S0=S, S_out=S, return_state=True)
    qs, ks, vs, os = [q], [k], [v], [o]
    for t in range(cut, l):
        # a column of the fused projection: rows of one token, L * width apart
        q, k, v = fw.norm_in(*(part(z, t, t + 1) for z in (q_in, k_in, v_in)))
        o = fw.gated_decode_step(S, q[:, :, 0], k[:, :, 0], v[:, :, 0], la[:, :, t].contiguous())
        y = fw.norm_out(o[:, :, None], x["w"], part(gate, t, t + 1), residual=part(x["res"], t, t + 1))
        ref = bo.norm_out(_np(o)[:, :, None], _np(x["w"]), _np(part(gate, t, t + 1)), "silu",
                          _np(part(x["res"], t, t + 1)))
        assert np.all(np.abs(_np(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-5)
        for a, b in ((qs, q), (ks, k), (vs, v), (os, o[:, :, None])):
            a.append(b)
    ro, rS = bo.gated_recurrence(*(_np(torch.cat(z, 2)) for z in (qs, ks, vs)), _np(la), _np(x["S0"]))
    _close(torch.cat(os, 2), ro, 1e-5)
    _close(S, rS, 1e-5)
