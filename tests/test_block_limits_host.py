"""Size limits of the norms' and the gated recurrence's entry points, before any HIP call
(fake, never-dereferenced pointers)."""
import os

import pytest

import weight_recurrent_memory_amd as fw
from weight_recurrent_memory_amd import binding

pytestmark = pytest.mark.cpu

UNSUPPORTED = 2
P = [(i + 1) << 42 for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        from weight_recurrent_memory_amd import build_lib
        build_lib.build()
    return fw.load_library()


@pytest.mark.parametrize("heads", [1 << 27, 1 << 29, (1 << 31) - 1])
def test_heads_of_the_norms(lib, heads):
    """A workgroup's rows (4 to 16 tokens of every head) are counted in 32 bits."""
    ld = heads * 16
    assert lib.falcon_norm_in(1, heads, 1, 16, 16, 0, P[0], ld, P[1], ld, P[2], ld, 1e-6, P[3], P[4],
                              P[5], None) == UNSUPPORTED
    assert lib.falcon_norm_in_bwd(1, heads, 1, 16, 16, 0, P[0], ld, P[1], ld, 1e-6, P[2], P[3], P[4],
                                  P[5], ld, P[6], ld, P[7], ld, None) == UNSUPPORTED
    assert lib.falcon_norm_out(1, heads, 1, 16, 0, P[0], P[1], P[2], ld, 0, P[3], ld, 1.0, 1e-6, P[4],
                               ld, None) == UNSUPPORTED
    assert lib.falcon_norm_out_bwd(1, heads, 1, 16, 0, P[0], P[1], P[2], ld, 0, 1.0, 1e-6, P[3], ld,
                                   P[4], P[5], ld, P[6], P[7], 1 << 20, None) == UNSUPPORTED
