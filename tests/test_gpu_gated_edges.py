"""The gated recurrence where it can go wrong: finite log decays that are resets, documents
of very different size in one sequence, entries that are not finite, padded batches.

Tolerances as derived in test_gpu_gated.py, u = 2^-24.
"""
import numpy as np
import pytest

from oracle import block_oracle as bo
from test_gpu_gated import TYPES, U, _factor, _gpu, _inputs, _np, _up  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import weight_recurrent_memory_amd as fw  # noqa: E402


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("reset", [-1001.0, -1000.0, -200.0, -110.0, -105.0])
@pytest.mark.parametrize("dk,dv,cut,L", [(32, 32, 50, 100), (64, 64, 1, 65), (128, 64, 700, 2500),
                                         (16, 128, 1023, 1025)])
def test_a_finite_reset_keeps_documents_apart(dtype, reset, dk, dv, cut, L):
    """Two documents, the loss of the first a millionth of the second's: the first one's
    dlog_a to rounding of its own sums (test_gpu_gated's bound of dlog_a over its tokens
    alone), exactly 0 at the border, where the true value is below 1e-45 times the states."""
    B, H = 1, 2
    x = _inputs(60, B, H, L, dk, dv, dtype)
    x["log_a"][:, :, cut] = reset
    dO = np.random.default_rng(61).standard_normal((B, H, L, dv))
    dO[:, :, :cut] *= 1e-6
    dO = _up(dO)
    got = _np(fw.gated_bwd_chunk(x["q"], x["k"], x["v"], x["log_a"], dO, S0=x["S0"])["dlog_a"])
    assert not got[:, :, cut].any()
    first = [_np(x[n])[:, :, :cut] for n in ("q", "k", "v", "log_a")]
    dO1, S0 = _np(dO)[:, :, :cut], _np(x["S0"])
    ref = bo.gated_backward(*first, dO1, S0)["dlog_a"]
    size = bo.gated_backward(*[np.abs(y) for y in first[:3]], first[3], np.abs(dO1), np.abs(S0))
    rc = np.sum(np.abs(first[0]) * size["dq"], -1) + np.sum(np.abs(first[1]) * size["dk"], -1)
    behind = np.cumsum(rc[..., ::-1], -1)[..., ::-1]
    tol = (_factor(L, dk, dv) + max(dk, dv)) * U * (behind + np.max(size["dlog_a"], -1, keepdims=True))
    bad = ~(np.abs(got[:, :, :cut] - ref) <= tol)
    assert not bad.any(), "%d off, worst %g times the tolerance" % (
        bad.sum(), np.nanmax(np.abs(got[:, :, :cut] - ref)[bad] / tol[bad]))


def _forward_size(x):
    """float64 outputs and the absolute sums of their terms, entries that are not finite
    among them."""
    with np.errstate(invalid="ignore", over="ignore"):
        a = [_np(x[n]) for n in ("q", "k", "v", "log_a", "S0")]
        ab = [None if y is None else np.abs(y) for y in a]
        ab[3] = a[3]
        return bo.gated_recurrence(*a), bo.gated_recurrence(*ab)


def _meets_where_finite(name, got, ref, size, factor):
    """Not finite exactly where the definition is not, and its value elsewhere."""
    got, fin = _np(got), np.isfinite(ref)
    assert np.array_equal(np.isfinite(got), fin), "%s: %d not finite, %d expected" % (
        name, (~np.isfinite(got)).sum(), (~fin).sum())
    if fin.any():
        tol = factor * U * np.maximum(size, 1e-6 * np.mean(size[np.isfinite(size)]))
        bad = fin & ~(np.abs(np.where(fin, got, 0) - np.where(fin, ref, 0)) <= tol)
        assert not bad.any(), "%s: %d off" % (name, bad.sum())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv,chains,L", [(64, 64, 3, 200), (16, 16, 2, 70), (128, 128, 2, 130), (32, 64, 128, 100),
                                            (128, 64, 130, 80), (64, 64, 2, 1500), (128, 128, 20, 900)])
@pytest.mark.parametrize("where", ["q", "k", "v", "log_a", "S0"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite_reaches_only_what_reads_it(dtype, dk, dv, chains, L, where, value):
    """One entry in two chains (the middle of a chunk, the last token): earlier tokens,
    other columns and other chains as if it were not there."""
    x = _inputs(62, 1, chains, L, dk, dv, dtype, start=True)
    for chain, t in ((0, 40 + 64 * (L // 128)), (chains - 1, L - 1)):
        if where == "S0":
            x["S0"][0, chain, 3, 5] = value
        elif where == "log_a":
            x["log_a"][0, chain, t] = value
        else:
            x[where][0, chain, t, 9] = value
    (ro, rS), (ao, aS) = _forward_size(x)
    for ws in ("auto", None):
        o, S = fw.gated_fwd_chunk(x["q"], x["k"], x["v"], x["log_a"], S0=x["S0"], return_state=True, workspace=ws)
        _meets_where_finite("o", o, ro, ao, _factor(L, dk, dv))
        _meets_where_finite("S", S, rS, aS, _factor(L, dk, dv))
    state = x["S0"].clone()
    o2 = fw.gated_fwd_chunk(x["q"], x["k"], x["v"], x["log_a"], S0=state, S_out=state, workspace=None)
    for a, b in ((o, o2), (S, state)):
        assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) and torch.equal(a.isnan(), b.isnan())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 32)])
def test_padded_batch(dtype, dk, dv):
    """Rows behind a sequence's last token may hold anything."""
    lengths = [1, 63, 64, 65, 100, 129, 130]
    x = _inputs(63, len(lengths), 2, 130, dk, dv, dtype, start=False)
    for b, n in enumerate(lengths):
        for m in ("q", "k", "v", "log_a"):
            x[m][b, :, n:] = float("nan")
    o = fw.gated_fwd_chunk(x["q"], x["k"], x["v"], x["log_a"])
    for b, n in enumerate(lengths):
        one = {m: t if t is None else t[b:b + 1, :, :n] for m, t in x.items()}
        (ro, _), (ao, _) = _forward_size(one)
        _meets_where_finite("o of %d" % n, o[b:b + 1, :, :n], ro, ao, _factor(n, dk, dv))


def test_nothing_is_left_behind():
    """A call on finite inputs between calls on others gives its bits, eager and captured."""
    x = _inputs(64, 1, 4, 500, 64, 64, torch.bfloat16)
    bad = {n: t.clone() for n, t in x.items()}
    bad["v"][0, 1, 333, 7] = float("inf")
    run = lambda y: fw.gated_fwd_chunk(y["q"], y["k"], y["v"], y["log_a"], S0=y["S0"])  # noqa: E731
    want, want_bad = run(x).clone(), run(bad).nan_to_num(7.0)
    assert torch.equal(run(x), want)
    bound = {n: t.clone() for n, t in x.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = run(bound)
    for y, w in ((bad, want_bad), (x, want), (bad, want_bad), (x, want)):
        for n, t in bound.items():
            t.copy_(y[n])
        graph.replay()
        run(x)
        torch.cuda.synchronize()
        assert torch.equal(o.nan_to_num(7.0), w)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv,L", [(64, 64, 300), (128, 64, 300), (64, 64, 2100)])
@pytest.mark.parametrize("where", ["q", "k", "v", "dO"])
def test_reach_of_a_nan_in_the_gradients(dtype, dk, dv, L, where):
    """Beside what depends on it: the other outputs of its chunk, and dlog_a of 1024 tokens
    at most, not before the last reset.  What lies elsewhere keeps its bits."""
    x = _inputs(65, 1, 2, L, dk, dv, dtype, gate="mixed")
    t, reset = 64 * (L // 128) + 40, 64 * (L // 128) - 30
    x["log_a"][0, 0, reset] = -float("inf")
    dO = _up(np.random.default_rng(66).standard_normal((1, 2, L, dv)))
    run = lambda: fw.gated_bwd_chunk(x["q"], x["k"], x["v"], x["log_a"], dO, S0=x["S0"])  # noqa: E731
    want = run()
    (dO if where == "dO" else x[where])[0, 0, t, 3] = float("nan")
    got = run()
    first, last = t // 64 * 64, t // 64 * 64 + 64            # its chunk
    for n in want:
        assert torch.equal(got[n][0, 1], want[n][0, 1]), n   # the other chain
    g, w = ({n: r[n][0, 0] for n in r} for r in (got, want))
    keys = where in ("k", "v")         # they are read by later tokens, q and dO by earlier ones
    if keys:
        assert torch.equal(g["dq"][:first], w["dq"][:first])
        assert torch.equal(g["dk"][:t], w["dk"][:t]) and torch.equal(g["dv"][:t], w["dv"][:t])
        assert torch.equal(g["dk"][t + 1:], w["dk"][t + 1:]) and torch.equal(g["dv"][t + 1:], w["dv"][t + 1:])
        assert torch.equal(g["dS0"], w["dS0"])
        assert torch.equal(g["dlog_a"][:reset + 1], w["dlog_a"][:reset + 1])
    else:
        assert torch.equal(g["dq"][:t], w["dq"][:t]) and torch.equal(g["dq"][t + 1:], w["dq"][t + 1:])
        assert torch.equal(g["dk"][last:], w["dk"][last:]) and torch.equal(g["dv"][last:], w["dv"][last:])
        assert torch.equal(g["dlog_a"][last:], w["dlog_a"][last:])
    assert not all(bool(r.isfinite().all()) for r in g.values())
