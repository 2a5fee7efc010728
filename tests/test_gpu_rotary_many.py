"""rotary_in and its gradient over many tokens: from 4096 on a workgroup takes eight tokens, from
2^20 such tiles on several of them.  Precision as in test_gpu_rotary.py."""
import pytest

from oracle import delta_oracle as do
from test_gpu_rotary import _gpu, _inputs, _meets, _np, _rows  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import numpy as np  # noqa: E402
import weight_recurrent_memory_amd as fw  # noqa: E402


def _check(x, dtype, B, L, H, dk, dv, **kw):
    q, k, v = fw.rotary_in(x["q"], x["k"], x["v"], x["pos"], x["f"], **kw)
    f, pos = _np(x["f"]), x["pos"].cpu().numpy()
    for name, got, raw in (("q", q, x["q"]), ("k", k, x["k"])):
        ref = do.rotary_in(_np(raw), pos, f, **kw)
        _meets(name, got, ref, dtype, _rows(ref))
    assert torch.equal(v, x["v"].transpose(1, 2))
    dqi, dki, dvi = fw.rotary_in_bwd(x["q"], x["k"], x["dq"], x["dk"], x["dv"], x["pos"], x["f"], **kw)
    for name, got, raw, dy in (("dq_in", dqi, x["q"], x["dq"]), ("dk_in", dki, x["k"], x["dk"])):
        ref = do.rotary_in_backward(_np(raw), _np(dy), pos, f, **kw)
        size = 2 * np.swapaxes(_rows(_np(dy)), 1, 2) / _rows(_np(raw))
        _meets(name, got, ref, dtype, size)
    assert torch.equal(dvi, x["dv"].transpose(1, 2).to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pairs", ["half", "neighbours"])
@pytest.mark.parametrize("dk,dv,rot", [(16, 128, 16), (16, 16, 10), (32, 64, 20), (64, 64, 64), (64, 16, 24), (128, 128, 128),
                                       (128, 32, 20)])
@pytest.mark.parametrize("B,L,H", [(1, 4096, 1), (3, 1367, 2)])
def test_tiles_of_eight_tokens(dtype, pairs, dk, dv, rot, B, L, H):
    x = _inputs(70 + dk + rot, B, L, H, dk, dv, dtype, rot)
    # (a gradient is divided by its row's norm: of rows of 16 columns, none is near 0)
    for n in ("q", "k"):
        x[n][..., 0] = 1.0
    _check(x, dtype, B, L, H, dk, dv, pairs=pairs)


@pytest.mark.parametrize("pairs,rot", [("half", 10), ("neighbours", 16)])
def test_workgroups_of_several_tiles(pairs, rot):
    """More than 2^20 tiles: the rows of the second round, against a call of their own and the fp64 form."""
    first, more, d = 8 << 20, 4101, 16
    g = torch.Generator(device="cuda").manual_seed(71)
    p = torch.randn((1, first + more, 1, 3 * d), generator=g, device="cuda", dtype=torch.bfloat16)
    p[..., ::d] = 1.0
    q, k, v = p[..., :d], p[..., d:2 * d], p[..., 2 * d:]
    pos = torch.arange(first + more, device="cuda")[None]
    f = fw.rotary_frequencies(rot, device="cuda")
    got = fw.rotary_in(q, k, v, pos, f, pairs=pairs)
    last = lambda t: t[:, first:].contiguous()  # noqa: E731
    own = fw.rotary_in(last(q), last(k), last(v), last(pos), f, pairs=pairs)
    head = lambda t: t[:, :more].contiguous()  # noqa: E731
    early = fw.rotary_in(head(q), head(k), head(v), head(pos), f, pairs=pairs)
    for a, b, c in zip(got, own, early):
        assert torch.equal(a[:, :, first:], b) and torch.equal(a[:, :, :more], c)
    for a, raw in ((got[0], q), (got[1], k)):
        ref = do.rotary_in(_np(last(raw)), last(pos).cpu().numpy(), _np(f), pairs=pairs)
        _meets("rotary_in", a[:, :, first:], ref, torch.bfloat16, _rows(ref))
    dy = [t.float() for t in got]
    back = fw.rotary_in_bwd(q, k, *dy, pos, f, pairs=pairs)
    part = lambda t: t[:, :, first:].contiguous()  # noqa: E731
    own = fw.rotary_in_bwd(last(q), last(k), *(part(t) for t in dy), last(pos), f, pairs=pairs)
    for a, b in zip(back, own):
        assert torch.equal(a[:, first:], b)
    for a, raw, t in ((back[0], q, dy[0]), (back[1], k, dy[1])):
        ref = do.rotary_in_backward(_np(last(raw)), _np(part(t)), last(pos).cpu().numpy(), _np(f), pairs=pairs)
        size = 2 * np.swapaxes(_rows(_np(part(t))), 1, 2) / _rows(_np(last(raw)))
        _meets("rotary_in_bwd", a[:, first:], ref, torch.bfloat16, size)
