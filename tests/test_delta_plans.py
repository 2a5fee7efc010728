"""CPU: the mirror of the gated delta rule's plans (delta_util.py) agrees with the library, its GPU
cases reach every kernel that the plans can pick, and a chain is cut where the workgroups that its
segments' launches really have leave it a gain."""
import itertools
import os

import numpy as np
import pytest

import delta_util as du
from weight_recurrent_memory_amd import block_binding

pytestmark = pytest.mark.cpu

LIMITS = [(f32, dk, dv, chains, L) for f32 in (False, True) for dk in du.DIMS for dv in du.DIMS
          for chains in (1, 2, 9, 14, 26, 27, 28, 40, 85, 86, 128, 129) for L in (640, 704, 2048, 4096)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(block_binding.library_path()):
        from weight_recurrent_memory_amd import build_lib
        build_lib.build()
    return block_binding.load_library()


def test_plans_are_the_librarys(lib):
    r = np.random.default_rng(1)
    some = [(bool(r.integers(2)), int(r.choice(du.DIMS)), int(r.choice(du.DIMS)), int(r.integers(1, 300)),
             int(np.exp(r.uniform(0, np.log(40000))))) for _ in range(2000)]
    for f32, dk, dv, chains, L in du.PLAN_CASES + LIMITS + some:
        size = (1, chains, L, dk, dv, int(f32))
        assert lib.falcon_gated_delta_fwd_workspace_bytes(*size) == du.forward_plan(chains, L, dk, dv, f32)[2], size
        assert lib.falcon_gated_delta_bwd_workspace_bytes(*size) == du.backward_plan(chains, L, dk, dv, f32)[2], size


@pytest.mark.parametrize("plan,case,segs", [
    # in one round each, values narrow and wide
    (du.forward_plan, (28, 4096, 128, 32, True), 3), (du.forward_plan, (9, 4096, 128, 16, False), 8),
    (du.backward_plan, (9, 4096, 128, 16, False), 7), (du.backward_plan, (26, 4096, 64, 32, True), 3),
    (du.forward_plan, (4, 32771, 128, 128, False), 16), (du.backward_plan, (5, 4099, 128, 64, False), 11),
    # 84 segments of 3 workgroups, 33 of them on an XCD: a second round where a compute unit holds one
    (du.backward_plan, (28, 4096, 64, 16, True), 1), (du.backward_plan, (28, 4096, 64, 32, True), 1),
    (du.backward_plan, (28, 4096, 64, 32, False), 3), (du.backward_plan, (14, 4096, 128, 128, True), 3),
    # 60 segments of 8 workgroups of the main walk: two rounds
    (du.forward_plan, (20, 2048, 128, 128, True), 1), (du.forward_plan, (20, 2048, 128, 128, False), 3),
    (du.forward_plan, (12, 4096, 128, 128, True), 5),
    # saving less than six chunks
    (du.forward_plan, (27, 704, 64, 64, False), 1), (du.forward_plan, (2, 640, 64, 64, False), 5)])
def test_what_is_cut(plan, case, segs):
    assert plan(*case)[1] == segs


def test_cases_reach_every_kernel():
    """The main walks of each type, dk and number of state waves, whole and cut; the segments' first
    launch and the join of each type and dk with them."""
    fwd, bwd = set(), set()
    for f32, dk, dv, chains, L in du.PLAN_CASES:
        for plan, reached in ((du.forward_plan, fwd), (du.backward_plan, bwd)):
            waves, segs, _ = plan(chains, L, dk, dv, f32)
            reached.add((f32, dk, waves, segs > 1))
    both = (False, True)
    assert bwd == set(itertools.product(both, du.DIMS, (1, 2, 4), both))
    assert fwd == set(itertools.product(both, du.DIMS, (1, 2), both)) - {(True, 128, 2, False), (True, 128, 2, True)}
