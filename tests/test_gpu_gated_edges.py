"""The gated recurrence where it can go wrong: finite log decays that are resets, documents
of very different size in one sequence.

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
