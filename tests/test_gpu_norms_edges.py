"""norm_in, norm_out and their gradients where they can go wrong: eps = 0, workgroups that
walk several tiles, gates far from zero, rows that are not finite.

Tolerances as derived in test_gpu_norms.py: u = 2^-24, h = half a step of the output type.
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


def _meets(got, ref, tol):
    got, tol = _np(got), np.broadcast_to(tol, np.shape(ref))
    assert got.shape == np.shape(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%d off, worst %g times the tolerance" % (
        bad.sum(), np.nanmax(np.abs(got - ref)[bad] / np.maximum(tol[bad], 1e-300)))


def _heads_first(x):
    return np.swapaxes(x, 1, 2)


def _check_norm_out_bwd(o, w, dy, gate, kind, eps, adds=256):
    """adds: additions that a term of dweight passes."""
    dv, dtype = o.shape[-1], dy.dtype
    d = fw.norm_out_bwd(o, w, dy, gate, gate_kind=kind or "silu", scale=0.5, eps=eps)
    ref = bo.norm_out_backward(_np(o), _np(w), _np(dy), None if gate is None else _np(gate),
                               kind or "silu", 0.5, eps)
    on = _heads_first(_np(o))
    r = 1 / np.sqrt(np.mean(on * on, -1, keepdims=True) + eps)
    n, dz = np.abs(r * on), np.abs(0.5 * _np(dy))
    if gate is not None:
        g = _np(gate)
        sg = bo.activation("sigmoid", g)[0]
        slope = sg * (1 + np.abs(g)) if kind == "silu" else sg
        _meets(d["dgate"], ref["dgate"], HALF[dtype] * np.abs(ref["dgate"])
               + (dv / 2 + 32) * U * dz * np.abs(_np(w)) * n * slope)
        dz = dz * np.abs(bo.activation(kind, g)[0])
    _meets(d["dweight"], ref["dweight"], (adds + dv / 2 + 32) * U * np.sum(dz * n, axis=(0, 1, 2)))
    dn = dz * np.abs(_np(w))
    size = r * (dn + n * np.mean(n * dn, -1, keepdims=True))
    _meets(d["dO"], ref["dO"], _heads_first((3 * dv + 64) * U * size))


# tokens and heads that do not fill a tile or a workgroup's lane groups, and one that does
EPS0 = [(512, 1, 12, 64), (2, 17, 12, 16), (1, 1, 1, 128), (1, 4099, 3, 32), (1, 4096, 16, 64)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,H,d", EPS0)
@pytest.mark.parametrize("kind", ["silu", "sigmoid", None])
def test_eps_zero_norm_out_bwd(B, L, H, d, dtype, kind):
    o, w, dy = _rand(1, B, H, L, d, std=0.5), 1 + _rand(2, d, std=0.1), _rand(3, B, L, H, d, dtype=dtype)
    gate = _rand(4, B, L, H, d, dtype=dtype) if kind else None
    _check_norm_out_bwd(o, w, dy, gate, kind, 0.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,H,d", EPS0)
def test_eps_zero_forward_and_norm_in(B, L, H, d, dtype):
    x, k = _rand(5, B, L, H, d, dtype=dtype), _rand(6, B, L, H, d, dtype=dtype)
    q, kk, _ = fw.norm_in(x, k, eps=0.0)
    for got, y in ((q, x), (kk, k)):
        ref = bo.unit_rows(_heads_first(_np(y)), 0.0)
        _meets(got, ref, (HALF[dtype] + (d / 2 + 6) * U) * np.abs(ref))
    g = _rand(7, B, H, L, d)
    for got, y in zip(fw.norm_in_bwd(x, k, g, g, eps=0.0), (x, k)):
        y, gg = _np(y), _heads_first(_np(g))
        r = 1 / np.sqrt(np.sum(y * y, -1, keepdims=True))
        ref, n = bo.unit_rows_backward(y, gg, 0.0), np.abs(r * y)
        size = r * (np.abs(gg) + n * np.sum(n * np.abs(gg), -1, keepdims=True))
        _meets(got, ref, HALF[dtype] * np.abs(ref) + (3 * d + 24) * U * size)
    o, w = _rand(8, B, H, L, d, std=0.5), 1 + _rand(9, d, std=0.1)
    y = fw.norm_out(o, w, x, scale=0.5, eps=0.0)
    ref = bo.norm_out(_np(o), _np(w), _np(x), "silu", None, 0.5, 0.0)
    _meets(y, ref, (HALF[dtype] + (d / 2 + 25) * U) * np.abs(ref))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["silu", "sigmoid"])
def test_gates_far_from_zero(kind, dtype):
    """A saturated gate's slope to float32 rounding of itself (a sigmoid's is e^-|g|):
    16u of s and 1 - s each beside the row's (d / 2 + 6) u; silu's 1 + g (1 - s) has terms
    of both signs, which count by their sizes."""
    L, d = 640, 64
    g = torch.linspace(-80, 80, L * d, device="cuda").view(1, L, 1, d).to(dtype)
    o, w, dy = _rand(10, 1, 1, L, d), 1 + _rand(11, d, std=0.1), _rand(12, 1, L, 1, d, dtype=dtype)
    got = fw.norm_out_bwd(o, w, dy, g, gate_kind=kind)["dgate"]
    on = _heads_first(_np(o))
    z = _np(dy) * _np(w) * on / np.sqrt(np.mean(on * on, -1, keepdims=True) + 1e-6)
    e = np.exp(-np.abs(_np(g)))
    s, rest = np.where(_np(g) >= 0, 1, e) / (1 + e), np.where(_np(g) >= 0, e, 1) / (1 + e)
    slope = s * rest if kind == "sigmoid" else s * (1 + _np(g) * rest)
    size = s * rest if kind == "sigmoid" else s * (1 + np.abs(_np(g)) * rest)
    _meets(got, z * slope, HALF[dtype] * np.abs(z * slope) + (d / 2 + 38) * U * np.abs(z) * size + 2.0 ** -126)


@pytest.mark.parametrize("B,L,H,d", [(3, 8195, 1, 16), (2, 20001, 2, 64)])
def test_workgroups_of_several_tiles(B, L, H, d):
    """dweight over more tiles than norm_out_bwd has workgroups (16384 tokens of 8): a term
    passes a lane's rows (under 16), 128 lane groups and 2048 workgroups' parts 32 at a time."""
    o, w = _rand(13, B, H, L, d, std=0.5), 1 + _rand(14, d, std=0.1)
    dy, gate = _rand(15, B, L, H, d, dtype=torch.bfloat16), _rand(16, B, L, H, d, dtype=torch.bfloat16)
    _check_norm_out_bwd(o, w, dy, gate, "silu", 1e-6)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("B,L,H,d", [(2, 17, 12, 16), (1, 4100, 3, 128)])
def test_a_row_that_is_not_finite_stays_by_itself(B, L, H, d, value, dtype):
    """Every other row keeps its bits; only dweight, the sum over all rows, has it too."""
    b, t, h = B - 1, L // 2, H - 1
    def calls(row):
        """Outputs and the place of the row in each, for a row of an input set to `value`."""
        q, k, v = (_rand(20 + i, B, L, H, d, dtype=dtype) for i in range(3))
        o, w, g = _rand(23, B, H, L, d), 1 + _rand(24, d, std=0.1), _rand(25, B, H, L, d)
        for n, x in (("q", q), ("v", v)):
            if row == n:
                x[b, t, h, 3] = value
        for n, x in (("o", o), ("g", g)):
            if row == n:
                x[b, h, t, 3] = value
        yield from zip("qkv", fw.norm_in(q, k, v))
        yield from zip(("dq", "dk", "dv"), fw.norm_in_bwd(q, k, g, g, g))
        yield "y", fw.norm_out(o, w, q, residual=v)
        for n, x in fw.norm_out_bwd(o, w, v, q).items():
            yield n, x
    clean = {n: x.clone() for n, x in calls(None)}
    for row in "qvog":
        touched = 0
        for n, x in calls(row):
            if n == "dweight":
                continue
            ref = clean[n]
            head_major = n in ("q", "k", "v", "dO")
            x, ref = ((y if head_major else y.transpose(1, 2)).clone() for y in (x, ref))
            touched += not bool(x[b, h, t].isfinite().all())
            x[b, h, t] = ref[b, h, t] = 0
            assert torch.equal(x, ref), (row, n)
        assert touched
