"""norm_in, norm_out and their gradients on the GPU against the fp64 forms.

Tolerances, u = 2^-24 (float32), h = half a step of the output type relative to the
value (bf16 2^-8, float32 2^-24):
  a sum of d squares is off by at most (d + 1) u of itself, its rsqrt by half of that
  plus 2u: r has a relative error of at most (d / 2 + 4) u.  An entry of q adds one
  product: e_r = (d / 2 + 6) u of its value.  Gradients r (g - y (y . g)): the dot
  product is off by at most (2d + 8) u sum |y g| (rounded products, d sums, the error of
  y twice), so an entry by (3d + 24) u r (|g_i| + |y_i| sum |y g|).  An activation and
  its slope add at most 16u of their own size, the slope counted as the sum of its terms'
  absolute values.  dweight: the terms' own error plus one u of the absolute sum for each
  addition on the way (rows of a lane, lane groups, workgroups: under 256 here).
"""
import numpy as np
import pytest

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import weight_recurrent_memory_amd as fw  # noqa: E402

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fw.load_library()


def _np(t):
    return t.detach().double().cpu().numpy()


def _rand(seed, *shape, dtype=torch.float32, std=1.0):
    r = np.random.default_rng(seed)
    return torch.from_numpy((std * r.standard_normal(shape)).astype(np.float32)).cuda().to(dtype)


def _projection(seed, B, L, H, dk, dv, dtype, pad=0):
    """q, k, v views of one fused projection, rows `pad` elements longer than needed."""
    w = H * (2 * dk + dv)
    p = _rand(seed, B, L, w + pad, dtype=dtype)
    if pad:
        p = p.as_strided((B, L, w), (L * (w + pad), w + pad, 1))
    cut = lambda a, n, d: p[..., a:a + n * d].view(B, L, n, d) if not pad else \
        p[..., a:a + n * d].as_strided((B, L, n, d), (L * (w + pad), w + pad, d, 1),
                                       p.storage_offset() + a)  # noqa: E731
    return cut(0, H, dk), cut(H * dk, H, dk), cut(2 * H * dk, H, dv)


def _meets(got, ref, tol):
    got, tol = _np(got), np.broadcast_to(tol, np.shape(ref))
    assert got.shape == np.shape(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%d off, worst %g times the tolerance" % (
        bad.sum(), np.nanmax(np.abs(got - ref)[bad] / np.maximum(tol[bad], 1e-300)))


def _heads_first(x):
    return np.swapaxes(x, 1, 2)


SHAPES = [  # B, L, H, dk, dv
    (1, 1, 1, 16, 16), (1, 1, 5, 128, 32), (7, 1, 3, 64, 64), (2, 17, 3, 32, 128),
    (1, 65, 12, 64, 16), (3, 1500, 1, 16, 64), (1, 4099, 2, 128, 128),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("pad", [0, 24])
def test_norm_in(shape, dtype, pad):
    B, L, H, dk, dv = shape
    q_in, k_in, v_in = _projection(1, B, L, H, dk, dv, dtype, pad)
    k_in[0, 0] = 0                                   # a row of zeros stays zero
    q, k, v = fw.norm_in(q_in, k_in, v_in, eps=1e-6)
    for got, x in ((q, q_in), (k, k_in)):
        ref = bo.unit_rows(_heads_first(_np(x)), 1e-6)
        _meets(got, ref, (HALF[dtype] + (dk / 2 + 6) * U) * np.abs(ref))
    assert torch.equal(v, v_in.transpose(1, 2))
    assert not k[0, :, 0].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fused", [False, True])
def test_norm_in_bwd(shape, dtype, fused):
    B, L, H, dk, dv = shape
    q_in, k_in, v_in = _projection(2, B, L, H, dk, dv, dtype)
    dq, dkk, dvv = _rand(3, B, H, L, dk), _rand(4, B, H, L, dk), _rand(5, B, H, L, dv)
    out = _projection(6, B, L, H, dk, dv, dtype) if fused else None
    got = fw.norm_in_bwd(q_in, k_in, dq, dkk, dvv, eps=1e-6, out=out)
    for d, x, g in ((got[0], q_in, dq), (got[1], k_in, dkk)):
        x, g = _np(x), _heads_first(_np(g))
        ref = bo.unit_rows_backward(x, g, 1e-6)
        r = 1 / np.sqrt(np.sum(x * x, -1, keepdims=True) + 1e-6)
        y = r * x
        size = r * (np.abs(g) + np.abs(y) * np.sum(np.abs(y * g), -1, keepdims=True))
        _meets(d, ref, HALF[dtype] * np.abs(ref) + (3 * dk + 24) * U * size)
    _meets(got[2], _heads_first(_np(dvv)), HALF[dtype] * np.abs(_heads_first(_np(dvv))))
    if fused:
        assert all(a is b for a, b in zip(got, out))


def test_norm_in_without_values():
    q_in, k_in, _ = _projection(7, 2, 5, 3, 32, 32, torch.bfloat16)
    q, k, v = fw.norm_in(q_in, k_in)
    q2, k2, _ = fw.norm_in(q_in, k_in, q_in)
    assert v is None and torch.equal(q, q2) and torch.equal(k, k2)
    dq = _rand(8, 2, 3, 5, 32)
    a, b, c = fw.norm_in_bwd(q_in, k_in, dq, dq)
    a2, b2, _ = fw.norm_in_bwd(q_in, k_in, dq, dq, dq)
    assert c is None and torch.equal(a, a2) and torch.equal(b, b2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "sigmoid", None])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_out(shape, dtype, kind, residual):
    B, L, H, _, dv = shape
    gate, res, _ = _projection(9, B, L, H, dv, dv, dtype)
    gate = gate * 4 if kind and B == 1 else gate
    o, w = _rand(10, B, H, L, dv, std=0.5), 1 + _rand(11, dv, std=0.1)
    o[0, 0, 0] = 0
    g, z = (gate if kind else None), (res if residual else None)
    y = fw.norm_out(o, w, g, gate_kind=kind or "silu", residual=z, scale=0.7, eps=1e-6, dtype=dtype)
    s = float(np.float32(0.7))
    t = bo.norm_out(_np(o), _np(w), None if g is None else _np(g), kind or "silu", None, s, 1e-6)
    ref = t if z is None else _np(z) + t
    _meets(y, ref, (HALF[dtype] + U) * np.abs(ref) + (dv / 2 + 24) * U * np.abs(t))
    if residual:                                     # in place over the residual
        fw.norm_out(o, w, g, gate_kind=kind or "silu", residual=res, scale=0.7, out=res)
        assert torch.equal(res, y)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "sigmoid", None])
def test_norm_out_bwd(shape, dtype, kind):
    B, L, H, _, dv = shape
    gate, dy, dgate = _projection(12, B, L, H, dv, dv, dtype)
    o, w = _rand(13, B, H, L, dv, std=0.5), 1 + _rand(14, dv, std=0.1)
    o[0, 0, 0] = 0
    g = gate if kind else None
    d = fw.norm_out_bwd(o, w, dy, g, gate_kind=kind or "silu", scale=0.7, eps=1e-6,
                        dgate=dgate if kind else None)
    again = fw.norm_out_bwd(o, w, dy, g, gate_kind=kind or "silu", scale=0.7, eps=1e-6)
    assert all(torch.equal(d[n], again[n]) for n in d)
    s = float(np.float32(0.7))
    ref = bo.norm_out_backward(_np(o), _np(w), _np(dy), None if g is None else _np(g),
                               kind or "silu", s, 1e-6)
    on = _heads_first(_np(o))
    r = 1 / np.sqrt(np.mean(on * on, -1, keepdims=True) + 1e-6)
    n, dz = np.abs(r * on), np.abs(s * _np(dy))
    if kind:
        gg = _np(gate)
        act, _ = bo.activation(kind, gg)
        sg = bo.activation("sigmoid", gg)[0]
        slope = sg * (1 + np.abs(gg)) if kind == "silu" else sg
        _meets(d["dgate"], ref["dgate"], HALF[dtype] * np.abs(ref["dgate"])
               + (dv / 2 + 32) * U * dz * np.abs(_np(w)) * n * slope)
        dz = dz * np.abs(act)
    _meets(d["dweight"], ref["dweight"], (256 + dv / 2 + 32) * U * np.sum(dz * n, axis=(0, 1, 2)))
    dn = dz * np.abs(_np(w))
    size = r * (dn + n * np.mean(n * dn, -1, keepdims=True))
    _meets(d["dO"], ref["dO"], _heads_first((3 * dv + 64) * U * size))


def test_offsets_beyond_32_bits():
    """2^31 elements and more: the last tokens' rows, zeros before them."""
    L, H, d, n = (1 << 20) + 5, 16, 128, 9
    x = torch.zeros((1, L, H, d), device="cuda", dtype=torch.bfloat16)
    x[:, -n:] = _rand(50, 1, n, H, d, dtype=torch.bfloat16)
    q, k, _ = fw.norm_in(x, x)
    small = fw.norm_in(x[:, -n:].contiguous(), x[:, -n:].contiguous())
    assert torch.equal(q[:, :, -n:], small[0]) and torch.equal(k[:, :, -n:], small[1])
    assert not q[:, :, :1000].any() and not q[:, :, -2000:-n].any()
    del q, k
    o = torch.zeros((1, H, L, d), device="cuda")
    o[:, :, -n:] = _rand(51, 1, H, n, d)
    w = 1 + _rand(52, d, std=0.1)
    y = fw.norm_out(o, w, x)
    cut = o[:, :, -n:].contiguous(), w, x[:, -n:].contiguous()
    assert torch.equal(y[:, -n:], fw.norm_out(*cut)) and not y[:, :-n].any()
    got = fw.norm_out_bwd(o, w, y, x)
    ref = fw.norm_out_bwd(cut[0], w, y[:, -n:].contiguous(), cut[2])
    assert torch.equal(got["dO"][:, :, -n:], ref["dO"]) and torch.equal(got["dgate"][:, -n:], ref["dgate"])
    # other workgroups' zeros beside the same terms: the sums' order may differ
    assert torch.allclose(got["dweight"], ref["dweight"], rtol=1e-5, atol=1e-4)


def test_norm_out_gradient_against_differences():
    """The kernels' gradients along random directions against central differences of
    the fp64 definition: they agree to the differences' own error (about 1e-9) and the
    kernels' (dv + 64) u of the products' absolute sums."""
    B, L, H, dv = 2, 9, 3, 32
    o, w, gate, dy = (_rand(20 + i, *s) for i, s in enumerate(
        ((B, H, L, dv), (dv,), (B, L, H, dv), (B, L, H, dv))))
    d = fw.norm_out_bwd(o, w, dy, gate, scale=0.5, eps=1e-3)
    args = [_np(o), _np(w), _np(gate)]
    r = np.random.default_rng(30)
    for i, name in enumerate(("dO", "dweight", "dgate")):
        u = r.standard_normal(args[i].shape)

        def f(h):
            x = list(args)
            x[i] = x[i] + h * u
            return np.sum(_np(dy) * bo.norm_out(*x, "silu", None, 0.5, 1e-3))
        want, have = (f(1e-5) - f(-1e-5)) / 2e-5, np.sum(_np(d[name]) * u)
        assert abs(want - have) <= 1e-6 + (256 + dv + 64) * U * np.sum(np.abs(_np(d[name]) * u)) * 4


@pytest.mark.parametrize("N", [1, 512])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 128), (64, 64), (128, 16), (128, 128)])
@pytest.mark.parametrize("gate", [True, False])
def test_gated_decode_step(N, dtype, dk, dv, gate):
    """Three steps in place.  A state entry: a rounded product, a rounded product and a
    sum, exp off by 2u: 5u of the absolute values a step.  o: two dot products of dk
    terms, (dk + 8) u of their absolute values beside the state's error."""
    H = 3
    S = _rand(40, N, H, dv, dk, std=0.3)
    ref, size = _np(S), np.abs(_np(S))
    for step in range(3):
        q, k, v = (_rand(41 + 3 * step + i, N, H, d, dtype=dtype) for i, d in enumerate((dk, dk, dv)))
        log_a = -_rand(60 + step, N, H).abs() if gate else None
        if gate:
            log_a[0, 0] = -float("inf")
        o = fw.gated_decode_step(S, q, k, v, log_a)
        cut = lambda x: _np(x)[:, :, None]  # noqa: E731
        la = None if log_a is None else _np(log_a)[:, :, None]
        want, ref = bo.gated_recurrence(cut(q), cut(k), cut(v), la, ref)
        aq, size = bo.gated_recurrence(np.abs(cut(q)), np.abs(cut(k)), np.abs(cut(v)), la, size)
        _meets(o, want[:, :, 0], (dk + 8 + 5 * (step + 1)) * U * aq[:, :, 0])
        _meets(S, ref, 5 * (step + 1) * U * size)
