"""Every kernel of the gated delta rule's sequence form (type, sizes, state waves, whole and cut)
against the rule in float64, to the precision of delta_util.py."""
import pytest

import delta_util as du
from test_gpu_delta import _check_backward, _check_forward, _gpu  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("case", du.PLAN_CASES, ids=str)
def test_kernels(case):
    f32, dk, dv, chains, L = case
    x = du.inputs(torch, 40 + dk + dv, 1, chains, L, dk, dv, torch.float32 if f32 else torch.bfloat16, gate="resets")
    _check_forward(x)
    _check_backward(x)


@pytest.mark.parametrize("f32,dk,dv,chains,L", [(False, 64, 16, 27, 1300), (True, 64, 32, 24, 1300), (True, 128, 32, 28, 1300),
                                                (True, 128, 16, 9, 1030), (False, 128, 32, 9, 1030)])
def test_segments_of_many_chains(f32, dk, dv, chains, L):
    """Without decay and half of the keys without a step, where a segment hands most on."""
    x = du.inputs(torch, 41, 1, chains, L, dk, dv, torch.float32 if f32 else torch.bfloat16, gate="none", beta="zero")
    _check_forward(x)
    _check_backward(x)
