"""Pins of the fp64 forms of the gated recurrence and the norms: central differences
along random directions, the resumed and the reset sequence, the library's own
inner-product rule as a special case."""
import numpy as np
import pytest

from oracle import block_oracle as bo
from oracle import falcon_oracle as fo

pytestmark = pytest.mark.cpu


def _inputs(seed, B=2, H=2, L=9, dk=4, dv=3):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((B, H, L, dk)), k=r.standard_normal((B, H, L, dk)),
                v=r.standard_normal((B, H, L, dv)), log_a=-r.random((B, H, L)),
                S0=r.standard_normal((B, H, dv, dk))), r


def _difference(f, x, u, h=1e-5):
    # central: error h^2 f''' / 6 plus 1e-16 |f| / h, both below 1e-9 of order-one values
    return (f(x + h * u) - f(x - h * u)) / (2 * h)


@pytest.mark.parametrize("name,grad", [("q", "dq"), ("k", "dk"), ("v", "dv"), ("log_a", "dlog_a"),
                                       ("S0", "dS0")])
def test_gated_gradients_against_differences(name, grad):
    x, r = _inputs(1)
    dO = r.standard_normal(x["v"].shape)
    dS = r.standard_normal(x["S0"].shape)
    d = bo.gated_backward(x["q"], x["k"], x["v"], x["log_a"], dO, x["S0"], dS)

    def loss(y):
        z = dict(x)
        z[name] = y
        o, S = bo.gated_recurrence(**z)
        return np.sum(o * dO) + np.sum(S * dS)
    u = r.standard_normal(x[name].shape)
    assert abs(_difference(loss, x[name], u) - np.sum(d[grad] * u)) < 1e-7 * max(1, np.abs(d[grad]).sum())


def test_gated_resumed_sequence():
    x, _ = _inputs(2)
    o, S = bo.gated_recurrence(**x)
    cut = lambda a, b: {n: x[n][:, :, a:b] for n in ("q", "k", "v", "log_a")}  # noqa: E731
    o1, S1 = bo.gated_recurrence(**cut(0, 4), S0=x["S0"])
    o2, S2 = bo.gated_recurrence(**cut(4, 9), S0=S1)
    assert np.array_equal(np.concatenate([o1, o2], 2), o) and np.array_equal(S2, S)


def test_gated_reset_is_a_fresh_sequence():
    x, _ = _inputs(3)
    x["log_a"][:, :, 5] = -np.inf
    o, S = bo.gated_recurrence(**x)
    o2, S2 = bo.gated_recurrence(*(x[n][:, :, 5:] for n in ("q", "k", "v", "log_a")))
    assert np.array_equal(o[:, :, 5:], o2) and np.array_equal(S, S2)


def test_gated_meets_the_inner_product_rule():
    """Falcon-1A with unit keys, eps 0, the same step's pairing: eta = beta, decay
    1 - beta lambda, write beta v k^T."""
    x, _ = _inputs(4)
    k = x["k"] / np.linalg.norm(x["k"], axis=-1, keepdims=True)
    o, S, _ = fo.falcon_recurrence(3, x["q"], k, x["v"], beta=0.5, lam=0.2, eps=0.0, same_step=True)
    o2, S2 = bo.gated_recurrence(x["q"], k, 0.5 * x["v"], np.full(x["log_a"].shape, np.log(0.9)))
    assert np.allclose(o, o2, rtol=1e-12, atol=1e-12) and np.allclose(S, S2, rtol=1e-12, atol=1e-12)


def test_unit_rows_gradient_against_differences():
    r = np.random.default_rng(5)
    x, dy, u = (r.standard_normal((3, 4, 5)) for _ in range(3))
    d = bo.unit_rows_backward(x, dy, 1e-3)
    assert abs(_difference(lambda y: np.sum(bo.unit_rows(y, 1e-3) * dy), x, u) - np.sum(d * u)) < 1e-8


@pytest.mark.parametrize("kind", ["silu", "sigmoid", None])
def test_norm_out_gradients_against_differences(kind):
    r = np.random.default_rng(6)
    o, gate = r.standard_normal((2, 3, 4, 5)), r.standard_normal((2, 4, 3, 5))
    w, dy = r.standard_normal(5), r.standard_normal((2, 4, 3, 5))
    g = None if kind is None else gate
    d = bo.norm_out_backward(o, w, dy, g, kind or "silu", 0.7, 1e-3)

    def loss(o, w, g):
        return np.sum(dy * bo.norm_out(o, w, g, kind or "silu", dy, 0.7, 1e-3))
    for i, (x, name) in enumerate(((o, "dO"), (w, "dweight"), (gate, "dgate"))):
        if name == "dgate" and kind is None:
            continue
        u = r.standard_normal(x.shape)
        args = [o, w, g]

        def f(y):
            z = list(args)
            z[i] = y
            return loss(*z)
        assert abs(_difference(f, x, u) - np.sum(d[name] * u)) < 1e-8 * max(1, np.abs(d[name]).sum())
