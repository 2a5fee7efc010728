"""Every kernel of the gated recurrence (type, sizes, block of rows or columns, whole and cut)
against the recurrence in float64, to the precision of gated_util.py."""
import numpy as np
import pytest

import gated_util as gu
from test_gpu_gated import _gpu, _inputs, _up  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import weight_recurrent_memory_amd as fw  # noqa: E402


def _heads(chains):
    """batch, heads of a number of chains."""
    return next((chains // h, h) for h in (16, 8, 5, 3, chains) if chains % h == 0)


def _case(seed, f32, dk, dv, chains, L):
    B, H = _heads(chains)
    return _inputs(seed, B, H, L, dk, dv, torch.float32 if f32 else torch.bfloat16, gate="mixed")


@pytest.mark.parametrize("case", gu.FORWARD_CASES, ids=str)
def test_forward_kernels(case):
    x = _case(70, *case)
    o, S = fw.gated_fwd_chunk(x["q"], x["k"], x["v"], x["log_a"], S0=x["S0"], return_state=True)
    ro, rS, _ = gu.recurrence(torch, **x)
    errors = dict(o=gu.off(o, ro), S=gu.off(S, rS))
    print(errors)
    assert max(errors.values()) <= gu.FORWARD, errors


@pytest.mark.parametrize("case", gu.BACKWARD_CASES, ids=str)
def test_backward_kernels(case):
    """dlog_a is a difference of sums of up to 1024 terms, each to float32 rounding: 2e-5 of
    its own size, as in test_gpu_gated.py."""
    x = _case(71, *case)
    r = np.random.default_rng(72)
    dO, dS = _up(r.standard_normal(x["v"].shape)), _up(0.3 * r.standard_normal(x["S0"].shape))
    got = fw.gated_bwd_chunk(x["q"], x["k"], x["v"], x["log_a"], dO, S0=x["S0"], dS_L=dS)
    want = gu.gradients(torch, dO=dO, dS_L=dS, **x)
    errors = {n: gu.off(got[n], want[n]) for n in want}
    print(errors)
    assert errors.pop("dlog_a") <= 2e-5
    assert max(errors.values()) <= gu.GRADIENT, errors
