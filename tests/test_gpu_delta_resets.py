"""Finite log decays around the smallest normal float32, 2^-126 = e^-87.34: below it a token is a
reset, in the sequence form, its gradients and the decode step alike.  The state before the token is of
size 2^120, so that a decay of e^-90 that counts would show.

At e^-86 and e^-87 (no resets) a decayed score's three bf16 parts end at bf16's least step, 2^-133: a
score P_ts across the token, and an entry of T, is off by up to 2^-134.  In the forward both meet u_s
of the tokens before, of the state's size: at most 2^-134 sum_s ||u_s|| twice in every later token's
outputs, and in the state.  In the gradients they meet dO behind the token: du and R before it are off
by 2^-134 (||dO|| + ||dS_L||) for P, T and the parts of R's update (roundings point either way), and for
P and T together: four times.  dv and dS0 hold that; dk, dbeta and dlog_a multiply it by what a unit
key reads of the state before, ||S0|| / sqrt(dk), and dq's u has the forward's error.  With tokens
behind it their decays bring the product below 2^-126, where it counts as 0: 2^-126 in the place of
2^-134.
"""
import math

import pytest

import delta_util as du

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import weight_recurrent_memory_amd as fw  # noqa: E402
from weight_recurrent_memory_amd import block_binding  # noqa: E402

AT = 3
NAMES = ("q", "k", "v", "beta", "log_a")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    block_binding.load_library()


def _inputs(dtype, L, value):
    """(inputs, the same with -inf where the token is a reset)."""
    x = du.inputs(torch, 50, 1, 2, L, 16, 32, dtype)
    x["S0"] = x["S0"] * 2.0 ** 120
    x["log_a"][:, :, :AT] = -0.01
    x["log_a"][:, :, AT] = value
    x["dO"][:, :, :AT] = 0.0
    y = dict(x, log_a=x["log_a"].clone())
    if value < -126 * math.log(2.0):
        y["log_a"][:, :, AT] = -float("inf")
    return x, y


def _step(L):
    """What a product of decays across the token is off by where the token is no reset."""
    return 2.0 ** (-134 if L == AT + 1 else -126)


def _least(x, errs):
    """sum_s ||u_s|| twice, of the tokens before the one at AT, times that."""
    return 2 * _step(x["q"].shape[2]) * sum(du.norm(x["beta"][:, :, s, None].double() * errs[s]) for s in range(AT))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L", [4, 70])
@pytest.mark.parametrize("value", [-86.0, -87.0, -88.0, -90.0, -103.0, -105.0, -500.0, -1000.0, -1e30])
def test_reset_of_a_finite_log_decay(dtype, L, value):
    x, y = _inputs(dtype, L, value)
    ro, rS, _, errs = du.recurrence(torch, y)
    least = _least(x, errs) if value > -87.2 else 0.0
    o, S = fw.gated_delta_fwd_chunk(*(x[n] for n in NAMES), S0=x["S0"], return_state=True)
    err = du.norm(o[:, :, AT:].double() - ro[:, :, AT:])
    assert err <= du.FORWARD * du.norm(ro[:, :, AT:]) + (L - AT) ** 0.5 * least
    assert du.norm(S.double() - rS) <= du.FORWARD * du.norm(rS) + least
    S = x["S0"].clone()
    for t in range(L):
        o = fw.gated_delta_decode_step(S, *(x[n][:, :, t].contiguous() for n in NAMES))
        if t >= AT:
            assert du.off(o, ro[:, :, t]) <= du.FORWARD, t
    assert du.off(S, rS) <= du.FORWARD


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L", [4, 70])
@pytest.mark.parametrize("value", [-86.0, -88.0, -90.0, -105.0, -1000.0, -1e30])
def test_gradients_at_and_before_it(dtype, L, value):
    """dlog_a and dbeta are differences, of terms as in test_gpu_delta.py; what is 0 behind the reset's
    back is 0 (tokens before it, whose outputs have no gradient here)."""
    x, y = _inputs(dtype, L, value)
    got = fw.gated_delta_bwd_chunk(*(x[n] for n in NAMES), x["dO"], S0=x["S0"], dS_L=x["dS_L"])
    ref = du.gradients(torch, y)
    vdv = (x["v"].double() * ref["dv"]).sum(-1)
    terms = dict(dlog_a=8 * (du.norm((x["q"].double() * ref["dq"]).sum(-1)) + du.norm(vdv)),
                 dbeta=du.norm(vdv / x["beta"].double().clamp(min=0.1)))
    if value > -87.2:
        behind = 4 * _step(L) * (du.norm(x["dO"]) + du.norm(x["dS_L"]))
        least = {n: behind * du.norm(x["S0"]) / 4 for n in ("dk", "dbeta", "dlog_a")}
        least.update(dv=behind, dS0=behind, dq=_least(x, du.recurrence(torch, y)[3]) * du.norm(x["dO"]))
    else:
        least = {}
    for n in got:
        err = du.norm(got[n].double() - ref[n])
        bound = du.GRADIENT * (du.norm(ref[n]) + terms.get(n, 0.0)) + least.get(n, 0.0)
        assert err <= bound, (n, err, bound, du.norm(ref[n]))
        if value < -126 * math.log(2.0) and n != "dS0":
            assert torch.all(got[n][:, :, :AT] == 0.0), n
    if value < -126 * math.log(2.0):
        assert torch.all(got["dlog_a"][:, :, AT] == 0.0) and torch.all(got["dS0"] == 0.0)
