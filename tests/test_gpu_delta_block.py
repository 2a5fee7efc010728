"""A block as it is used: rotary_in, the gated delta rule and norm_out, forward and backward,
against the fp64 forms; captured and replayed; then served token by token."""
import numpy as np
import pytest

from oracle import block_oracle as bo
from oracle import delta_oracle as do

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import weight_recurrent_memory_amd as fw  # noqa: E402

B, L, H, DK, DV, ROT = 2, 150, 3, 32, 64, 16
WIDTH = H * (2 * DK + 2 * DV)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, ref, rel):
    assert np.linalg.norm(_np(got) - ref) <= rel * np.linalg.norm(ref)


def _batch(seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return dict(p=rn(B, L, WIDTH).to(dtype), log_a=torch.nn.functional.logsigmoid(rn(B, H, L) + 3),
                beta=torch.sigmoid(rn(B, H, L)), w=1 + 0.1 * rn(DV), dy=rn(B, L, H, DV).to(dtype),
                S0=0.2 * rn(B, H, DV, DK), pos=(torch.arange(L, device="cuda") + 1000).repeat(B, 1),
                f=fw.rotary_frequencies(ROT, scaling="linear", factor=2.0, device="cuda"))


def _views(p):
    at, out = 0, []
    for d in (DK, DK, DV, DV):
        out.append(p[..., at:at + H * d].view(p.shape[0], p.shape[1], H, d))
        at += H * d
    return out


def _run(x):
    q_in, k_in, v_in, gate = _views(x["p"])
    q, k, v = fw.rotary_in(q_in, k_in, v_in, x["pos"], x["f"])
    o, S = fw.gated_delta_fwd_chunk(q, k, v, x["beta"], x["log_a"], S0=x["S0"], return_state=True)
    y = fw.norm_out(o, x["w"], gate)
    n = fw.norm_out_bwd(o, x["w"], x["dy"], gate)
    d = fw.gated_delta_bwd_chunk(q, k, v, x["beta"], x["log_a"], n["dO"], S0=x["S0"])
    dp = torch.empty_like(x["p"])
    dq_in, dk_in, dv_in, dgate = _views(dp)
    fw.rotary_in_bwd(q_in, k_in, d["dq"], d["dk"], d["dv"], x["pos"], x["f"], out=(dq_in, dk_in, dv_in))
    dgate.copy_(n["dgate"])
    return dict(y=y, S=S, dp=dp, dweight=n["dweight"], dbeta=d["dbeta"], dlog_a=d["dlog_a"], dS0=d["dS0"])


def test_block_against_the_oracle():
    x = _batch(1, torch.float32)
    got = _run(x)
    q_in, k_in, v_in, gate = (_np(t) for t in _views(x["p"]))
    pos, f = x["pos"].cpu().numpy(), _np(x["f"])
    q, k = do.rotary_in(q_in, pos, f), do.rotary_in(k_in, pos, f)
    v = np.swapaxes(v_in, 1, 2)
    b, la, S0, w = (_np(x[n]) for n in ("beta", "log_a", "S0", "w"))
    o, S = do.delta_recurrence(q, k, v, b, la, S0)
    _close(got["y"], bo.norm_out(o, w, gate), 1e-5)
    _close(got["S"], S, 1e-5)
    n = bo.norm_out_backward(o, w, _np(x["dy"]), gate)
    d = do.delta_backward(q, k, v, b, la, n["dO"], S0)
    ref = [do.rotary_in_backward(q_in, d["dq"], pos, f), do.rotary_in_backward(k_in, d["dk"], pos, f),
           np.swapaxes(d["dv"], 1, 2), n["dgate"]]
    for t, r in zip(_views(got["dp"]), ref):
        _close(t, r, 1e-5)
    for m in ("dbeta", "dlog_a", "dS0"):
        _close(got[m], d[m], 1e-5)
    _close(got["dweight"], n["dweight"], 1e-5)


def test_block_captured_and_replayed():
    x = _batch(2, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = _run(x)
    for seed in (3, 4, 5):
        for n, t in _batch(seed, torch.bfloat16).items():
            x[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in kept.items()}
        want = _run(x)
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_block_served_token_by_token():
    """A prompt, then single tokens: the same outputs as the whole sequence at once."""
    x = _batch(6, torch.bfloat16)
    q_in, k_in, v_in, gate = _views(x["p"])
    q, k, v = fw.rotary_in(q_in, k_in, v_in, x["pos"], x["f"])
    o = fw.gated_delta_fwd_chunk(q, k, v, x["beta"], x["log_a"])
    cut = 140
    head = lambda t: t[:, :, :cut].contiguous()  # noqa: E731
    _, S = fw.gated_delta_fwd_chunk(head(q), head(k), head(v), head(x["beta"]), head(x["log_a"]), return_state=True)
    for t in range(cut, L):
        one = slice(t, t + 1)
        q1, k1, v1 = fw.rotary_in(q_in[:, one], k_in[:, one], v_in[:, one], x["pos"][:, one].contiguous(), x["f"])
        assert torch.equal(q1[:, :, 0], q[:, :, t]) and torch.equal(k1[:, :, 0], k[:, :, t])
        o1 = fw.gated_delta_decode_step(S, q1[:, :, 0], k1[:, :, 0], v1[:, :, 0], x["beta"][:, :, t].contiguous(),
                                        x["log_a"][:, :, t].contiguous())
        _close(o1, _np(o[:, :, t]), 1e-5)
        y1 = fw.norm_out(o1[:, :, None], x["w"], gate[:, one])
        assert y1.shape == (B, 1, H, DV)
