"""Refusals of the gated delta rule's and the rotary positions' entry points, before any HIP
call (fake, never-dereferenced pointers) and in the binding; the exported names; the
frequencies."""
import math
import os
import re
import subprocess

import pytest

import weight_recurrent_memory_amd as fw
from weight_recurrent_memory_amd import block_binding

pytestmark = pytest.mark.cpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = 1, 2
P = [0x100000000 + 0x10000000 * i for i in range(20)]
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(block_binding.library_path()):
        from weight_recurrent_memory_amd import build_lib
        build_lib.build()
    return block_binding.load_library()


def _call(fn, defaults, over):
    assert set(over) <= set(defaults), over
    return fn(*{**defaults, **over}.values(), None)


def test_exported_names(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "falcon_block.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(falcon_\w+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", block_binding.library_path()], capture_output=True,
                         text=True, check=True).stdout
    assert {x for x in (line.split()[-1] for line in out.splitlines()) if "falcon" in x} == declared
    assert all(hasattr(lib, n) for n in declared)


FWD = dict(batch=2, heads=3, seqlen=100, dk=64, dv=64, dtype=0, q=P[0], k=P[1], v=P[2], beta=P[3], log_a=P[4],
           S0=P[5], o=P[6], S_out=P[7], ws=P[8], wsb=1 << 28)
BWD = dict(batch=2, heads=3, seqlen=100, dk=64, dv=64, dtype=0, q=P[0], k=P[1], v=P[2], beta=P[3], log_a=P[4],
           S0=P[5], dO=P[6], dS_L=P[7], dq=P[8], dk_=P[9], dv_=P[10], dbeta=P[11], dlog_a=P[12], dS0=P[13],
           ws=P[14], wsb=1 << 28)
DEC = dict(nseq=2, heads=3, dk=64, dv=64, dtype=0, S=P[0], q=P[1], k=P[2], v=P[3], beta=P[4], log_a=P[5], o=P[6])
SIZES = [(dict(heads=0), INVALID), (dict(dtype=2), INVALID), (dict(dv=48), UNSUPPORTED), (dict(dk=256), UNSUPPORTED)]
SEQ = SIZES + [(dict(batch=0), INVALID), (dict(seqlen=0), INVALID), (dict(seqlen=-5), INVALID),
               (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(beta=None), INVALID),
               (dict(ws=None), INVALID), (dict(wsb=100), INVALID), (dict(q=P[0] + 8), INVALID),
               (dict(beta=P[3] + 2), INVALID), (dict(log_a=P[4] + 1), INVALID),
               (dict(batch=1 << 16, seqlen=1 << 15), INVALID),
               (dict(batch=1 << 12, heads=1 << 12, seqlen=127, ws=1 << 60), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", SEQ + [
    (dict(o=None), INVALID), (dict(o=P[6] + 4), INVALID), (dict(ws=P[8] + 8), INVALID), (dict(o=P[0]), INVALID),
    (dict(S_out=P[6] + 256), INVALID), (dict(S_out=P[5] + 1024), INVALID), (dict(ws=P[3]), INVALID),
    (dict(ws=P[5]), INVALID), (dict(S_out=P[4]), INVALID),
])
def test_forward(lib, over, status):
    assert _call(lib.falcon_gated_delta_fwd_chunk, FWD, over) == status


@pytest.mark.parametrize("over,status", SEQ + [
    (dict(dO=None), INVALID), (dict(dq=None), INVALID), (dict(dk_=None), INVALID), (dict(dv_=None), INVALID),
    (dict(dbeta=None), INVALID), (dict(log_a=None), INVALID), (dict(dO=P[6] + 4), INVALID),
    (dict(dbeta=P[11] + 2), INVALID), (dict(dlog_a=P[12] + 3), INVALID), (dict(dq=P[0]), INVALID),
    (dict(dv_=P[6]), INVALID), (dict(dS0=P[5]), INVALID), (dict(dS0=P[7] + 64), INVALID), (dict(dlog_a=P[11]), INVALID),
    (dict(ws=P[8] + 64), INVALID), (dict(ws=P[14] + 4), INVALID),
])
def test_backward(lib, over, status):
    assert _call(lib.falcon_gated_delta_bwd_chunk, BWD, over) == status


@pytest.mark.parametrize("over,status", SIZES + [
    (dict(nseq=0), INVALID), (dict(S=None), INVALID), (dict(beta=None), INVALID), (dict(o=None), INVALID),
    (dict(q=P[1] + 2), INVALID), (dict(beta=P[4] + 2), INVALID), (dict(o=P[0] + 64), INVALID), (dict(o=P[5]), INVALID),
    (dict(S=P[4]), INVALID),
    (dict(nseq=1 << 18, heads=16, S=1 << 44, q=1 << 40, k=2 << 40, v=3 << 40, beta=4 << 40, log_a=5 << 40, o=6 << 40),
     UNSUPPORTED),
])
def test_decode(lib, over, status):
    assert _call(lib.falcon_gated_delta_decode_step, DEC, over) == status


# (batch, heads, L, dk, dv) just below 2^32 work-items of a launch, and just above: 12 for a value row of
# each chain (8 chains side by side) and 64 for a chunk in the forward; in the gradients 16 and 24 for a
# value row at dv of 32 and 16, and 256 for a chunk.
FORWARD_LIMITS = [((349525, 8, 1, 16, 128), (349526, 8, 1, 16, 128)), ((699050, 8, 64, 16, 64), (699051, 8, 64, 16, 64)),
                  ((2796202, 8, 1, 16, 16), (2796203, 8, 1, 16, 16)),
                  ((1, 4, (1 << 30) - 64, 16, 16), (1, 4, (1 << 30) - 63, 16, 16))]
BACKWARD_LIMITS = [((349525, 8, 1, 16, 128), (349526, 8, 1, 16, 128)), ((1048575, 8, 1, 16, 32), (1048576, 8, 1, 16, 32)),
                   ((1398101, 8, 1, 16, 16), (1398102, 8, 1, 16, 16)),
                   ((1, 15, 64 * 1118481, 16, 16), (1, 16, 64 * 1048576, 16, 16))]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("name,below,above", [("fwd", *x) for x in FORWARD_LIMITS] + [("bwd", *x) for x in BACKWARD_LIMITS])
def test_work_items_of_a_launch(lib, name, below, above, dtype):
    """A launch has fewer than 2^32 work-items: sizes beyond are unsupported, and not an error of the
    launch."""
    size = getattr(lib, "falcon_gated_delta_%s_workspace_bytes" % name)
    assert size(*below, dtype) > 0 and size(*above, dtype) == 0
    defaults = FWD if name == "fwd" else BWD
    over = dict(zip(("batch", "heads", "seqlen", "dk", "dv"), above), dtype=dtype, wsb=1 << 62)
    over.update({n: (i + 1) << 44 for i, n in enumerate(list(defaults)[6:-1])})
    call = getattr(lib, "falcon_gated_delta_%s_chunk" % name)
    assert _call(call, defaults, over) == UNSUPPORTED


def test_workspace_sizes(lib):
    for f in (lib.falcon_gated_delta_fwd_workspace_bytes, lib.falcon_gated_delta_bwd_workspace_bytes):
        assert f(0, 1, 1, 64, 64, 0) == f(1, 1, 1, 48, 64, 0) == f(1, 1, 0, 64, 64, 0) == 0
        assert f(1 << 12, 1 << 12, 127, 64, 64, 0) == 0
        assert 0 < f(1, 1, 1, 16, 16, 0) < f(1, 1, 65, 16, 16, 0)
    # every chunk's T: six operands of three planes
    assert lib.falcon_gated_delta_fwd_workspace_bytes(8, 12, 2048, 64, 64, 0) == 8 * 12 * 32 * 18432


ROT = dict(batch=2, heads=3, seqlen=8, dk=64, dv=64, dtype=0, q_in=P[0], ld_q=576, k_in=P[0] + 384, ld_k=576,
           v_in=P[0] + 768, ld_v=576, positions=P[1], freqs=P[2], rot=64, pairs=0, scale=1.0, normalize=1, eps=1e-6,
           q=P[3], k=P[4], v=P[5])
ROT_BWD = dict(batch=2, heads=3, seqlen=8, dk=64, dv=64, dtype=0, q_in=P[0], ld_q=576, k_in=P[0] + 384, ld_k=576,
               positions=P[1], freqs=P[2], rot=64, pairs=0, scale=1.0, normalize=1, eps=1e-6, dq=P[3], dk_=P[4],
               dv_=P[5], dq_in=P[6], ld_dq=576, dk_in=P[6] + 384, ld_dk=576, dv_in=P[6] + 768, ld_dv=576)
ROTATION = SIZES[:3] + [
    (dict(batch=0), INVALID), (dict(seqlen=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(q_in=None), INVALID), (dict(k_in=P[0] + 388), INVALID), (dict(ld_q=191), INVALID), (dict(ld_k=580), INVALID),
    (dict(positions=None), INVALID), (dict(freqs=None), INVALID), (dict(positions=P[1] + 4), INVALID),
    (dict(freqs=P[2] + 4), INVALID), (dict(rot=0), INVALID), (dict(rot=31), INVALID), (dict(rot=66), INVALID),
    (dict(pairs=2), INVALID), (dict(scale=INF), INVALID), (dict(normalize=2), INVALID), (dict(heads=1 << 27, seqlen=1,
     batch=1, dk=16, dv=16, rot=16, ld_q=1 << 31, ld_k=1 << 31, q_in=1 << 44, k_in=2 << 44), UNSUPPORTED)]


def _far(over):
    """Arguments of the largest sizes lie far apart."""
    if over.get("heads", 0) < 1 << 20:
        return over
    names = ("v_in", "q", "k", "v", "dq", "dk_", "dv_", "dq_in", "dk_in", "dv_in")
    far = {n: (5 + i) << 44 for i, n in enumerate(names)}
    return {**over, **far, "ld_v": 1 << 31, "ld_dq": 1 << 31, "ld_dk": 1 << 31, "ld_dv": 1 << 31}


@pytest.mark.parametrize("over,status", ROTATION + [
    (dict(q=None), INVALID), (dict(v=None), INVALID), (dict(v_in=None), INVALID), (dict(k=P[4] + 4), INVALID),
    (dict(q=P[0] + 1024), INVALID), (dict(q=P[4]), INVALID), (dict(k=P[1]), INVALID), (dict(v=P[2]), INVALID),
])
def test_rotary_in(lib, over, status):
    over = {n: v for n, v in _far(over).items() if n in ROT}
    assert _call(lib.falcon_rotary_in, ROT, over) == status


@pytest.mark.parametrize("over,status", ROTATION + [
    (dict(dq=None), INVALID), (dict(dk_in=None), INVALID), (dict(dv_=None), INVALID), (dict(dv_in=None), INVALID),
    (dict(dq=P[3] + 4), INVALID), (dict(ld_dq=100), INVALID), (dict(dk_in=P[6] + 368), INVALID),
    (dict(dq_in=P[0]), INVALID), (dict(dq_in=P[1]), INVALID), (dict(dq_in=P[3]), INVALID),
])
def test_rotary_in_bwd(lib, over, status):
    over = {n: v for n, v in _far(over).items() if n in ROT_BWD}
    assert _call(lib.falcon_rotary_in_bwd, ROT_BWD, over) == status


def test_binding_refuses_host_tensors_and_wrong_arguments(lib):
    torch = pytest.importorskip("torch")
    z = lambda *s: torch.zeros(s)  # noqa: E731
    q = z(1, 2, 4, 16)
    with pytest.raises(ValueError):
        fw.gated_delta_fwd_chunk(q, q, q, z(1, 2, 4))
    with pytest.raises(ValueError):
        fw.gated_delta_bwd_chunk(q, q, q, z(1, 2, 4), None, q)
    with pytest.raises(ValueError):
        fw.gated_delta_decode_step(z(1, 2, 16, 16), z(1, 2, 16), z(1, 2, 16), z(1, 2, 16), z(1, 2))
    with pytest.raises(ValueError):
        fw.rotary_in(q, q, q, torch.zeros(1, 2, dtype=torch.int64), fw.rotary_frequencies(16))
    with pytest.raises(ValueError):
        fw.rotary_in_bwd(q, q, q, q, q, torch.zeros(1, 2, dtype=torch.int64), fw.rotary_frequencies(16))


def test_frequencies():
    torch = pytest.importorskip("torch")
    f = fw.rotary_frequencies(8)
    assert f.dtype == torch.float64 and f.shape == (4,)
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    assert torch.equal(fw.rotary_frequencies(8, scaling="linear", factor=4.0), f / 4.0)
    b = fw.rotary_frequencies(8, scaling="base", factor=4.0)
    assert b[0] == 1.0 and abs(float(b[3]) - 0.001 / 4.0) < 1e-15
    t = fw.rotary_frequencies(8, scaling="by_turns", factor=4.0, original_length=2000, slow=1.0, fast=32.0)
    turns = 2000 * f / (2 * math.pi)                 # 318, 32 (31.8), 3.2, 0.3
    left = ((turns - 1.0) / 31.0).clamp(0, 1)
    assert torch.allclose(t, f * left + f / 4.0 * (1 - left)) and t[0] == f[0] and t[3] == f[3] / 4.0
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, base=-1.0), dict(rot=8, factor=0.0), dict(rot=8, scaling="x"),
                dict(rot=8, scaling="by_turns", factor=2.0), dict(rot=2, scaling="base", factor=2.0)):
        with pytest.raises(ValueError):
            fw.rotary_frequencies(**bad)
