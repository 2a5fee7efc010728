"""CPU: the gated recurrence's GPU cases reach every kernel that its plans can pick, the
mirror of those plans agrees with the library, and the precision asked for tells three bf16
planes of an operand from two."""
import itertools
import os

import numpy as np
import pytest

import gated_util as gu
import weight_recurrent_memory_amd as fw
from oracle import block_oracle as bo
from weight_recurrent_memory_amd import binding

pytestmark = pytest.mark.cpu


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        from weight_recurrent_memory_amd import build_lib
        build_lib.build()
    return fw.load_library()


def test_plans_are_the_librarys(lib):
    r = np.random.default_rng(1)
    some = [(bool(r.integers(2)), int(r.choice(gu.DIMS)), int(r.choice(gu.DIMS)), int(r.integers(1, 400)),
             int(np.exp(r.uniform(0, np.log(40000))))) for _ in range(2000)]
    for f32, dk, dv, chains, L in gu.FORWARD_CASES + gu.BACKWARD_CASES + some:
        size = (1, chains, L, dk, dv, int(f32))
        assert lib.falcon_gated_fwd_workspace_bytes(*size) == gu.forward_plan(chains, L, dk, dv, f32)[2], size
        assert lib.falcon_gated_bwd_workspace_bytes(*size) == gu.backward_plan(chains, L, dk, dv, f32)[2], size


def test_cases_reach_every_forward_kernel():
    """A kernel for each type, dk and block of value rows, walked whole and cut."""
    reached = set()
    for f32, dk, dv, chains, L in gu.FORWARD_CASES:
        block, segs, _ = gu.forward_plan(chains, L, dk, dv, f32)
        reached.add((f32, dk, block, segs > 1))
    assert reached == set(itertools.product((False, True), gu.DIMS, (16, 32, 64), (False, True)))


def test_cases_reach_every_backward_kernel():
    """A kernel for each type, dk and dv; with a size of 128, for each block of columns: of
    16, 32 and 64, the last not for bf16 at dk >= 64."""
    reached = set()
    for f32, dk, dv, chains, L in gu.BACKWARD_CASES:
        block, segs, _ = gu.backward_plan(chains, L, dk, dv, f32)
        reached.add((f32, dk, dv, block, segs > 1))
    want = set()
    for f32, dk, dv, cut in itertools.product((False, True), gu.DIMS, gu.DIMS, (False, True)):
        blocks = (0,) if max(dk, dv) <= 64 else (16, 32, 64) if f32 or dk < 64 else (16, 32)
        want |= {(f32, dk, dv, b, cut) for b in blocks}
    assert reached == want


def _bf16(x):
    """x rounded to bf16 (to nearest, ties to even), float64 in and out."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def _planes(x, n):
    """The value of x's first n bf16 planes."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    y = np.zeros_like(x)
    for _ in range(n):
        y = y + _bf16(x - y)
    return y


def _chunked(q, k, v, log_a, n):
    """The chunk form of one chain in float64, with scores and states (and the inputs, where
    they are float32) held in n planes."""
    L, C = q.shape[0], gu.C
    S, o = np.zeros((v.shape[1], k.shape[1])), np.empty_like(v)
    q, k, v = (_planes(x, n) for x in (q, k, v))
    for a in range(0, L, C):
        b = min(a + C, L)
        G = np.cumsum(log_a[a:b])
        D = np.tril(np.exp(G[:, None] - G[None, :]))
        P = _planes(q[a:b] @ k[a:b].T * D, n)
        o[a:b] = P @ v[a:b] + np.exp(G)[:, None] * (q[a:b] @ _planes(S, n).T)
        w = _planes(v[a:b] * np.exp(G[-1] - G)[:, None], n)
        S = np.exp(G[-1]) * S + w.T @ k[a:b]
    return o, S


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("d,L", [(16, 130), (64, 321), (128, 321)])
def test_precision_asked_tells_two_planes_from_three(f32, d, L):
    r = np.random.default_rng(d + L)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    q, k, v = unit(r.standard_normal((L, d))), unit(r.standard_normal((L, d))), r.standard_normal((L, d))
    q, k, v = (_planes(x, 3 if f32 else 1) for x in (q, k, v))
    log_a = -np.log1p(np.exp(-(2.0 * r.standard_normal(L) + 3.0)))
    o, S = (x[0, 0] for x in bo.gated_recurrence(*(x[None, None] for x in (q, k, v, log_a))))
    errors = {n: [gu.off(*x) for x in zip(_chunked(q, k, v, log_a, n), (o, S))] for n in (2, 3)}
    assert max(errors[3]) < gu.FORWARD / 4
    assert errors[2][0] > 1.2 * gu.GRADIENT and errors[2][1] > 1.2 * gu.FORWARD
