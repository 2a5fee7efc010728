"""Pins of the fp64 forms of the gated delta rule and of rotary positions: central
differences along random directions, resumed and reset sequences, the library's own
regression rule and the gated recurrence as special cases, what a rotation keeps."""
import numpy as np
import pytest

from oracle import block_oracle as bo
from oracle import delta_oracle as do
from oracle import falcon_oracle as fo

pytestmark = pytest.mark.cpu


def _inputs(seed, B=2, H=2, L=9, dk=4, dv=3):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((B, H, L, dk)), k=bo.unit_rows(r.standard_normal((B, H, L, dk)), 0.0),
                v=r.standard_normal((B, H, L, dv)), beta=r.random((B, H, L)), log_a=-r.random((B, H, L)),
                S0=r.standard_normal((B, H, dv, dk))), r


@pytest.mark.parametrize("name,grad", [("q", "dq"), ("k", "dk"), ("v", "dv"), ("beta", "dbeta"),
                                       ("log_a", "dlog_a"), ("S0", "dS0")])
def test_gradients_against_differences(name, grad):
    x, r = _inputs(1)
    dO, dS = r.standard_normal(x["v"].shape), r.standard_normal(x["S0"].shape)
    d = do.delta_backward(x["q"], x["k"], x["v"], x["beta"], x["log_a"], dO, x["S0"], dS)

    def loss(y):
        o, S = do.delta_recurrence(**{**x, name: y})
        return np.sum(o * dO) + np.sum(S * dS)
    u, h = r.standard_normal(x[name].shape), 1e-5
    # central: error h^2 f''' / 6 plus 1e-16 |f| / h, both below 1e-8 of order-one values
    got = (loss(x[name] + h * u) - loss(x[name] - h * u)) / (2 * h)
    assert abs(got - np.sum(d[grad] * u)) < 1e-7 * max(1, np.abs(d[grad]).sum())


def test_resumed_and_reset_sequence():
    x, _ = _inputs(2)
    o, S = do.delta_recurrence(**x)
    cut = lambda a, b: {n: x[n][:, :, a:b] for n in ("q", "k", "v", "beta", "log_a")}  # noqa: E731
    o1, S1 = do.delta_recurrence(**cut(0, 4), S0=x["S0"])
    o2, S2 = do.delta_recurrence(**cut(4, 9), S0=S1)
    assert np.array_equal(np.concatenate([o1, o2], 2), o) and np.array_equal(S2, S)
    x["log_a"][:, :, 4] = -np.inf
    o, S = do.delta_recurrence(**x)
    o2, S2 = do.delta_recurrence(**cut(4, 9))
    assert np.allclose(o[:, :, 4:], o2, atol=1e-14) and np.allclose(S, S2, atol=1e-14)


def test_regression_rule_is_a_special_case():
    """Unit keys, eps = 0, lambda = 0, the same step's key: eta_t = beta_t, no decay."""
    x, _ = _inputs(3)
    o, S = do.delta_recurrence(x["q"], x["k"], x["v"], x["beta"], None, x["S0"])
    ref = fo.falcon_recurrence(fo.FALCON_1, x["q"], x["k"], x["v"], beta=1.0, beta_t=x["beta"], lam=0.0,
                               eps=0.0, S0=x["S0"], same_step=True)
    assert np.allclose(o, ref[0], atol=1e-12) and np.allclose(S, ref[1], atol=1e-12)


def test_small_steps_are_the_gated_recurrence():
    """beta -> 0 with v / beta: the erase vanishes, to first order in beta."""
    x, _ = _inputs(4)
    b = 1e-9 * x["beta"]
    o, S = do.delta_recurrence(x["q"], x["k"], x["v"] / b[..., None], b, x["log_a"])
    ro, rS = bo.gated_recurrence(x["q"], x["k"], x["v"], x["log_a"])
    assert np.allclose(o, ro, atol=1e-7) and np.allclose(S, rS, atol=1e-7)


@pytest.mark.parametrize("pairs", ["half", "neighbours"])
def test_turn_depends_on_differences_only(pairs):
    r = np.random.default_rng(5)
    q, k = r.standard_normal((2, 1, 2, 1, 10))
    f = np.array([1.0, 0.3, 0.01])
    dot = lambda a, b: np.sum(do.turn(q, np.full((1, 1), a), f, pairs) * do.turn(k, np.full((1, 1), b), f, pairs))  # noqa: E731
    assert abs(dot(3, 7) - dot(103, 107)) < 1e-12
    assert abs(dot(0, 0) - np.sum(q * k)) < 1e-12


@pytest.mark.parametrize("pairs", ["half", "neighbours"])
@pytest.mark.parametrize("normalize", [True, False])
def test_rotary_gradient_against_differences(pairs, normalize):
    r = np.random.default_rng(6)
    x, dy, u = r.standard_normal((2, 5, 3, 8)), r.standard_normal((2, 3, 5, 8)), r.standard_normal((2, 5, 3, 8))
    pos, f = r.integers(0, 1000, (2, 5)), np.array([1.0, 0.1, 0.003])
    kw = dict(pairs=pairs, scale=1.2, normalize=normalize)
    h = 1e-6
    d = (np.sum(do.rotary_in(x + h * u, pos, f, **kw) * dy) - np.sum(do.rotary_in(x - h * u, pos, f, **kw) * dy)) / (2 * h)
    assert abs(d - np.sum(do.rotary_in_backward(x, dy, pos, f, **kw) * u)) < 1e-6
