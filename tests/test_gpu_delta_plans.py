"""Every kernel of the gated delta rule's sequence form (type, sizes, state waves, whole and cut)
against the rule in float64, to the precision of delta_util.py."""
import pytest

import delta_util as du
from test_gpu_delta import _check_backward, _check_forward, _gpu  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import weight_recurrent_memory_amd as fw  # noqa: E402


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


def test_as_many_chains_as_a_launch_takes():
    """One token of 2796200 chains at dv = 128, the last size below 2^32 work-items of the walk: o is
    beta (k . q) v.  (T of one chunk a chain takes 51 GB.)"""
    B, H = 349525, 8
    g = torch.Generator(device="cuda").manual_seed(42)
    rn = lambda d: torch.randn((B, H, 1, d), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, beta = rn(16) * 0.25, rn(16) * 0.25, rn(128), torch.rand((B, H, 1), generator=g, device="cuda")
    o = fw.gated_delta_fwd_chunk(q, k, v, beta)
    for at in range(0, B, 65536):
        part = slice(at, at + 65536)
        want = (beta[part].double() * (k[part].double() * q[part].double()).sum(-1))[..., None] * v[part].double()
        assert du.off(o[part], want) <= du.FORWARD, at
    del o
    torch.cuda.empty_cache()
