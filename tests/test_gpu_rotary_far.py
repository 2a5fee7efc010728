"""rotary_in and its gradient at positions up to 2^53, against angles of 100 digits; precision as in
test_gpu_rotary.py.  (An angle that is one float64 product is off by half a unit at 2^53.)"""
from decimal import Decimal, getcontext

import numpy as np
import pytest

from oracle.block_oracle import unit_rows, unit_rows_backward
from test_gpu_rotary import _gpu, _inputs, _meets, _np, _rows  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import weight_recurrent_memory_amd as fw  # noqa: E402

POSITIONS = [2 ** 53 - 1, -(2 ** 53 - 1), 2 ** 52 + 12345, -(2 ** 50 + 777), 2 ** 45 + 1, 10 ** 12 + 7, 2 ** 33, 123456789]


def _pi():
    """16 atan(1/5) - 4 atan(1/239)."""
    def atan(n):
        x, total, k = Decimal(1) / n, Decimal(0), 0
        while abs(x) > Decimal(10) ** -115:
            total += (x if k % 2 == 0 else -x) / (2 * k + 1)
            x, k = x / (n * n), k + 1
        return total
    return 16 * atan(5) - 4 * atan(239)


def _angles(positions, freqs):
    """position * frequency to within pi of 0, float64."""
    getcontext().prec = 120
    turn = 2 * _pi()
    assert str(turn / 2).startswith("3.14159265358979323846264338327950288")
    out = np.empty((len(positions), len(freqs)))
    for i, p in enumerate(positions):
        for j, f in enumerate(freqs):
            a = Decimal(p) * Decimal(float(f))
            out[i, j] = float(a - (a / turn).to_integral_value() * turn)
    return out


def _turn(x, angle, pairs, sign):
    """x [B,H,L,d], its first columns turned by angle [L, rot / 2]."""
    y, n = x.copy(), angle.shape[1]
    i, j = (slice(0, n), slice(n, 2 * n)) if pairs == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    c, s = np.cos(angle), sign * np.sin(angle)
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    return y


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pairs", ["half", "neighbours"])
@pytest.mark.parametrize("rot,base", [(64, 10000.0), (16, 500000.0)])
def test_positions_to_2_53(dtype, pairs, rot, base):
    L = len(POSITIONS)
    x = _inputs(60, 1, L, 3, 64, 64, dtype, rot)
    x["f"] = fw.rotary_frequencies(rot, base, device="cuda")
    pos = torch.tensor([POSITIONS], device="cuda")
    angle = _angles(POSITIONS, _np(x["f"]))
    q, k, _ = fw.rotary_in(x["q"], x["k"], None, pos, x["f"], pairs=pairs)
    for got, raw in ((q, x["q"]), (k, x["k"])):
        ref = _turn(np.swapaxes(unit_rows(_np(raw), 1e-6), 1, 2), angle, pairs, 1.0)
        _meets("rotary_in", got, ref, dtype, _rows(ref))
    dq, dk, _ = fw.rotary_in_bwd(x["q"], x["k"], x["dq"], x["dk"], None, pos, x["f"], pairs=pairs)
    for got, raw, dy in ((dq, x["q"], x["dq"]), (dk, x["k"], x["dk"])):
        back = np.swapaxes(_turn(_np(dy), angle, pairs, -1.0), 1, 2)
        size = 2 * np.swapaxes(_rows(_np(dy)), 1, 2) / _rows(_np(raw))
        _meets("rotary_in_bwd", got, unit_rows_backward(_np(raw), back, 1e-6), dtype, size)
