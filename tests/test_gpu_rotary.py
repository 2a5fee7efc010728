"""rotary_in and its gradient against the fp64 form.  A float32 result is wrong by the norm's
sums and products, an angle's fraction of a turn rounded to float32 (2^-25 turns = 1.9e-7 of a
column, 3 u) and the rotation's three operations: below 16 u of the row's norm, u = 2^-24; a
bf16 result also by half a step, 2^-8 of the value (with the float32 error in it)."""
import numpy as np
import pytest

from oracle import delta_oracle as do

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import weight_recurrent_memory_amd as fw  # noqa: E402

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _np(t):
    return t.detach().double().cpu().numpy()


def _meets(name, got, ref, dtype, size):
    """|got - ref| <= 16 u of the row's size, and half a step of the value in bf16."""
    got = _np(got)
    assert got.shape == ref.shape
    step = torch.finfo(dtype).eps / 2
    tol = 16 * U * size + step * (np.abs(ref) + 16 * U * size)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d off, worst %g" % (name, bad.sum(), np.max(np.abs(got - ref)[bad] / tol[bad]))


def _rows(x):
    return np.linalg.norm(x, axis=-1, keepdims=True)


def _inputs(seed, B, L, H, dk, dv, dtype, rot, far=4096, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    p = rn(B, L, H * (2 * dk + dv)).to(dtype)
    cut = lambda a, d: p[..., a:a + H * d].view(B, L, H, d)  # noqa: E731
    pos = torch.randint(-far, far, (B, L), generator=g, device=device)
    return dict(q=cut(0, dk), k=cut(H * dk, dk), v=cut(2 * H * dk, dv), pos=pos,
                f=fw.rotary_frequencies(rot, device=device), dq=rn(B, H, L, dk), dk=rn(B, H, L, dk), dv=rn(B, H, L, dv))


CASES = [(16, 2), (16, 8), (16, 16), (32, 8), (32, 20), (64, 48), (64, 64), (128, 24), (128, 96), (128, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk,rot", CASES)
@pytest.mark.parametrize("pairs", ["half", "neighbours"])
@pytest.mark.parametrize("normalize", [True, False])
def test_forward_and_backward(dtype, dk, rot, pairs, normalize):
    dv = {16: 64, 32: 16, 64: 32, 128: 128}[dk]
    for B, L, H in ((1, 1, 1), (2, 37, 3)):
        x = _inputs(dk + rot + L, B, L, H, dk, dv, dtype, rot)
        kw = dict(pairs=pairs, scale=1.25, normalize=normalize)
        q, k, v = fw.rotary_in(x["q"], x["k"], x["v"], x["pos"], x["f"], **kw)
        f, pos = _np(x["f"]), x["pos"].cpu().numpy()
        for name, got, raw in (("q", q, x["q"]), ("k", k, x["k"])):
            ref = do.rotary_in(_np(raw), pos, f, **kw)
            _meets(name, got, ref, dtype, _rows(ref))
        assert torch.equal(v, x["v"].transpose(1, 2))
        dqi, dki, dvi = fw.rotary_in_bwd(x["q"], x["k"], x["dq"], x["dk"], x["dv"], x["pos"], x["f"], **kw)
        for name, got, raw, dy in (("dq_in", dqi, x["q"], x["dq"]), ("dk_in", dki, x["k"], x["dk"])):
            ref = do.rotary_in_backward(_np(raw), _np(dy), pos, f, **kw)
            size = 1.25 * np.swapaxes(_rows(_np(dy)), 1, 2)
            if normalize:
                size = 2 * size / _rows(_np(raw))
            _meets(name, got, ref, dtype, size)
        assert torch.equal(dvi, x["dv"].transpose(1, 2).to(dtype))


def test_far_positions():
    """Positions of 10^6 and of 2^40: a float32 product would keep no fraction of a turn."""
    for at in (10 ** 6, 1 << 40):
        x = _inputs(5, 1, 64, 2, 64, 64, torch.float32, 64)
        pos = at + torch.arange(64, device="cuda")[None]
        q, _, _ = fw.rotary_in(x["q"], x["k"], None, pos, x["f"])
        # the oracle's own angle, a float64 product, is off by 2^-53 of itself
        ref = do.rotary_in(_np(x["q"]), pos.cpu().numpy(), _np(x["f"]))
        _meets("q", q, ref, torch.float32, _rows(ref) * (1 + at * 2.0 ** -52 / U))


def test_scores_depend_on_differences_of_positions():
    x = _inputs(6, 1, 50, 2, 32, 32, torch.float32, 32)
    pos = torch.arange(50, device="cuda")[None]
    dots = []
    for shift in (0, 12345):
        q, k, _ = fw.rotary_in(x["q"], x["k"], None, pos + shift, x["f"])
        dots.append(torch.matmul(q, k.transpose(-1, -2)))
    assert float((dots[0] - dots[1]).abs().max()) <= 64 * U       # two rows of 16 u each, both ways


@pytest.mark.parametrize("L", [1, 5000])
def test_zero_rows_eps_and_many_tokens(L):
    x = _inputs(7, 3, L, 2, 16, 16, torch.bfloat16, 16)
    x["q"][0, 0] = 0.0
    q, k, v = fw.rotary_in(x["q"], x["k"], x["v"], x["pos"], x["f"], eps=1e-3)
    assert torch.all(q[0, :, 0] == 0)
    ref = do.rotary_in(_np(x["k"]), x["pos"].cpu().numpy(), _np(x["f"]), eps=1e-3)
    _meets("k", k, ref, torch.bfloat16, _rows(ref))


def test_what_is_not_finite_stays_in_its_row():
    x = _inputs(8, 2, 40, 3, 32, 32, torch.bfloat16, 20)
    want = fw.rotary_in(x["q"], x["k"], x["v"], x["pos"], x["f"])
    x["q"][1, 7, 2, 3] = float("nan")
    q, k, v = fw.rotary_in(x["q"], x["k"], x["v"], x["pos"], x["f"])
    assert torch.equal(k, want[1]) and torch.isnan(q[1, 2, 7]).all()
    q[1, 2, 7] = want[0][1, 2, 7]
    assert torch.equal(q, want[0])


def test_outputs_given_views_of_one_buffer_and_streams():
    B, L, H, d = 2, 33, 3, 64
    x = _inputs(9, B, L, H, d, d, torch.bfloat16, 64)
    want = fw.rotary_in_bwd(x["q"], x["k"], x["dq"], x["dk"], x["dv"], x["pos"], x["f"])
    buf = torch.full((B, L, 3 * H * d + 16), 3.0, device="cuda", dtype=torch.bfloat16)
    out = tuple(buf[..., i * H * d:(i + 1) * H * d].view(B, L, H, d) for i in range(3))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fw.rotary_in_bwd(x["q"], x["k"], x["dq"], x["dk"], x["dv"], x["pos"], x["f"], out=out, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.all(buf[..., 3 * H * d:] == 3.0)
    q = torch.empty((B, H, L, d), device="cuda", dtype=torch.bfloat16)
    k, v = torch.empty_like(q), torch.empty_like(q)
    got = fw.rotary_in(x["q"], x["k"], x["v"], x["pos"], x["f"], out=(q, k, v))
    assert got[0] is q and torch.equal(q, fw.rotary_in(x["q"], x["k"], None, x["pos"], x["f"])[0])
