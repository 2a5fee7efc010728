"""Refusals of the norms' and the gated recurrence's entry points, before any HIP call
(fake, never-dereferenced pointers) and in the binding."""
import os

import pytest

import weight_recurrent_memory_amd as fw
from weight_recurrent_memory_amd import binding

pytestmark = pytest.mark.cpu

INVALID, UNSUPPORTED = 1, 2
P = [0x100000000 + 0x10000000 * i for i in range(16)]
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        from weight_recurrent_memory_amd import build_lib
        build_lib.build()
    return fw.load_library()


def _call(fn, defaults, over):
    a = dict(defaults)
    assert set(over) <= set(a), over
    a.update(over)
    return fn(*a.values(), None)


NORM_IN = dict(batch=2, heads=3, seqlen=8, dk=64, dv=64, dtype=0, q_in=P[0], ld_q=576,
               k_in=P[0] + 384, ld_k=576, v_in=P[0] + 768, ld_v=576, eps=1e-6, q=P[1], k=P[2],
               v=P[3])
NORM_IN_BWD = dict(batch=2, heads=3, seqlen=8, dk=64, dv=64, dtype=0, q_in=P[0], ld_q=576,
                   k_in=P[0] + 384, ld_k=576, eps=1e-6, dq=P[1], dk_=P[2], dv_=P[3], dq_in=P[4],
                   ld_dq=576, dk_in=P[4] + 384, ld_dk=576, dv_in=P[4] + 768, ld_dv=576)
NORM_OUT = dict(batch=2, heads=3, seqlen=8, dv=64, dtype=0, o=P[0], weight=P[1], gate=P[2],
                ld_gate=192, gate_kind=0, residual=P[3], ld_res=192, scale=1.0, eps=1e-6, y=P[4],
                ld_y=192)
NORM_OUT_BWD = dict(batch=2, heads=3, seqlen=8, dv=64, dtype=0, o=P[0], weight=P[1], gate=P[2],
                    ld_gate=192, gate_kind=0, scale=1.0, eps=1e-6, dy=P[3], ld_dy=192, dO=P[4],
                    dgate=P[5], ld_dgate=192, dweight=P[6], ws=P[7], wsb=1 << 20)
DECODE = dict(nseq=2, heads=3, dk=64, dv=64, dtype=0, S=P[0], q=P[1], k=P[2], v=P[3], log_a=P[4],
              o=P[5])

SIZES = [(dict(heads=0), INVALID), (dict(dtype=2), INVALID), (dict(dv=48), UNSUPPORTED)]
SEQ = SIZES + [(dict(batch=0), INVALID), (dict(seqlen=0), INVALID),
               (dict(batch=1 << 16, seqlen=1 << 15), INVALID), (dict(eps=-1.0), INVALID),
               (dict(eps=NAN), INVALID)]


@pytest.mark.parametrize("over,status", SEQ + [
    (dict(dk=256, ld_q=3 * 256, ld_k=3 * 256), UNSUPPORTED),
    (dict(q_in=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(v_in=None), INVALID),       # one without the other
    (dict(q_in=P[0] + 8), INVALID), (dict(k=P[2] + 4), INVALID),   # alignment
    (dict(ld_q=191), INVALID), (dict(ld_k=580), INVALID), (dict(ld_q=-576), INVALID),
    (dict(ld_v=1 << 41), INVALID),
    (dict(q=P[0] + 1024), INVALID), (dict(q=P[2]), INVALID),   # overlaps
])
def test_norm_in(lib, over, status):
    assert _call(lib.falcon_norm_in, NORM_IN, over) == status


@pytest.mark.parametrize("over,status", SEQ + [
    (dict(dq=None), INVALID), (dict(dk_in=None), INVALID), (dict(dv_=None), INVALID),
    (dict(dv_in=None), INVALID), (dict(dq=P[1] + 4), INVALID), (dict(dq_in=P[4] + 8), INVALID),
    (dict(ld_dq=100), INVALID),
    (dict(dk_in=P[4] + 368), INVALID),               # rows that reach into dq_in's
    (dict(dv_in=P[4] + 784), INVALID),               # rows that reach the next token's dq_in
    (dict(dk_in=P[4] + 384, ld_dk=584), INVALID),    # interleaved with another distance
    (dict(dq_in=P[0]), INVALID), (dict(dq_in=P[1]), INVALID),
])
def test_norm_in_bwd(lib, over, status):
    assert _call(lib.falcon_norm_in_bwd, NORM_IN_BWD, over) == status


@pytest.mark.parametrize("over,status", SEQ + [
    (dict(o=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID),
    (dict(gate_kind=2), INVALID), (dict(gate_kind=-1), INVALID), (dict(scale=INF), INVALID),
    (dict(weight=P[1] + 4), INVALID), (dict(y=P[4] + 8), INVALID), (dict(ld_gate=64), INVALID),
    (dict(y=P[0]), INVALID), (dict(y=P[1]), INVALID), (dict(y=P[2]), INVALID),
    (dict(y=P[3] + 16), INVALID), (dict(y=P[3], ld_y=200), INVALID),   # not exactly in place
])
def test_norm_out(lib, over, status):
    assert _call(lib.falcon_norm_out, NORM_OUT, over) == status


@pytest.mark.parametrize("over,status", SEQ + [
    (dict(dy=None), INVALID), (dict(dO=None), INVALID), (dict(dweight=None), INVALID),
    (dict(ws=None), INVALID), (dict(wsb=0), INVALID), (dict(ws=P[7] + 8), INVALID),
    (dict(gate=None), INVALID), (dict(dgate=None), INVALID), (dict(gate_kind=2), INVALID),
    (dict(scale=NAN), INVALID), (dict(dgate=P[2]), INVALID), (dict(dO=P[0]), INVALID),
    (dict(ws=P[4] + 64), INVALID), (dict(dweight=P[3]), INVALID), (dict(ld_dy=190), INVALID),
])
def test_norm_out_bwd(lib, over, status):
    assert _call(lib.falcon_norm_out_bwd, NORM_OUT_BWD, over) == status


def test_norm_out_bwd_workspace(lib):
    f = lib.falcon_norm_out_bwd_workspace_bytes
    assert f(1, 1, 64) == 64 * 4                     # one workgroup's part of dweight
    assert f(8, 2048, 64) == 2048 * 64 * 4
    assert f(0, 1, 64) == f(1, 1, 48) == f(1 << 16, 1 << 15, 64) == 0


@pytest.mark.parametrize("over,status", SIZES + [
    (dict(nseq=0), INVALID), (dict(dk=24), UNSUPPORTED), (dict(S=None), INVALID),
    (dict(o=None), INVALID), (dict(q=P[1] + 2), INVALID), (dict(log_a=P[4] + 2), INVALID),
    (dict(o=P[0] + 64), INVALID), (dict(o=P[4]), INVALID), (dict(S=P[2]), INVALID),
    (dict(nseq=1 << 18, heads=16, S=1 << 44, q=1 << 40, k=2 << 40, v=3 << 40, log_a=4 << 40,
          o=5 << 40), UNSUPPORTED),
])
def test_gated_decode_step(lib, over, status):
    assert _call(lib.falcon_gated_decode_step, DECODE, over) == status


def test_binding_refuses_host_tensors_and_odd_layouts():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 2, 3, 16)
    with pytest.raises(ValueError):
        fw.norm_in(x, x, x)
    with pytest.raises(ValueError):
        fw.norm_out(x, x[0, 0, 0])
    with pytest.raises(ValueError):
        fw.gated_decode_step(x, x[0], x[0], x[0])
    rows = fw.norms._rows
    ok = torch.zeros(2, 5, 96)[..., 48:].view(2, 5, 3, 16)
    assert rows(torch, "x", ok, (2, 5, 3, 16), torch.float32, ok.device)[1] == 96
    assert rows(torch, "x", ok[:, :1], (2, 1, 3, 16), torch.float32, ok.device)[1] == 480
    for bad in (ok.transpose(1, 2).contiguous().transpose(1, 2), ok[:, ::2], ok[..., ::2],
                ok[:, :, :1].expand(2, 5, 3, 16), ok[:1].expand(2, 5, 3, 16)):
        with pytest.raises(ValueError):
            rows(torch, "x", bad, tuple(bad.shape), torch.float32, bad.device)
    # a projection with one more column a head behind it: rows 3 elements off 16 bytes
    odd = torch.zeros(2, 5, 99)[..., :48].view(2, 5, 3, 16)
    shifted = torch.zeros(2 * 5 * 48 + 1)[1:].view(2, 5, 3, 16)
    for bad in (odd, shifted):
        with pytest.raises(ValueError, match="16"):
            rows(torch, "x", bad, (2, 5, 3, 16), torch.float32, bad.device)
    with pytest.raises(ValueError):
        fw.norms._gate_kind("relu")


FWD = dict(batch=2, heads=3, seqlen=8, dk=64, dv=64, dtype=0, q=P[0], k=P[1], v=P[2], log_a=P[3],
           S0=P[4], o=P[5], S_out=P[6], ws=P[7], wsb=0)
BWD = dict(batch=2, heads=3, seqlen=8, dk=64, dv=64, dtype=0, q=P[0], k=P[1], v=P[2], log_a=P[3],
           S0=P[4], dO=P[5], dS_L=P[6], dq=P[7], dk_=P[8], dv_=P[9], dlog_a=P[10], dS0=P[11],
           ws=P[12], wsb=1 << 20)


@pytest.mark.parametrize("over,status", SIZES + [
    (dict(batch=0), INVALID), (dict(seqlen=0), INVALID), (dict(batch=1 << 16, seqlen=1 << 15), INVALID),
    (dict(dk=24), UNSUPPORTED), (dict(q=None), INVALID), (dict(o=None), INVALID),
    (dict(k=P[1] + 8), INVALID), (dict(log_a=P[3] + 2), INVALID), (dict(ws=P[7] + 8), INVALID),
    (dict(o=P[0]), INVALID), (dict(o=P[3]), INVALID), (dict(S_out=P[2]), INVALID),
    (dict(S_out=P[4] + 64), INVALID),                # the start's state only exactly in place
    (dict(o=P[4]), INVALID), (dict(S_out=P[5]), INVALID),
    (dict(seqlen=2048, ws=P[5] + 4096, wsb=1 << 26), INVALID),   # workspace inside o
    (dict(batch=1 << 17, heads=16, seqlen=1, q=1 << 44, k=2 << 40, v=3 << 40, log_a=4 << 40,
          S0=5 << 40, o=6 << 40, S_out=7 << 40), UNSUPPORTED),
])
def test_gated_fwd_chunk(lib, over, status):
    assert _call(lib.falcon_gated_fwd_chunk, FWD, over) == status


@pytest.mark.parametrize("over,status", SIZES + [
    (dict(batch=0), INVALID), (dict(seqlen=-1), INVALID), (dict(dk=256), UNSUPPORTED),
    (dict(dO=None), INVALID), (dict(dq=None), INVALID), (dict(ws=None), INVALID),
    (dict(wsb=100), INVALID), (dict(ws=P[12] + 8), INVALID), (dict(log_a=None), INVALID),
    (dict(dO=P[5] + 4), INVALID), (dict(dq=P[0]), INVALID), (dict(dk_=P[7]), INVALID),
    (dict(dS0=P[4]), INVALID), (dict(dS0=P[6]), INVALID), (dict(dlog_a=P[10] + 2), INVALID), (dict(dlog_a=P[3]), INVALID),
    (dict(ws=P[9] + 64), INVALID),
    (dict(heads=512, batch=64, seqlen=1 << 17, q=1 << 45, k=2 << 45, v=3 << 45, log_a=4 << 45,
          S0=5 << 45, dO=6 << 45, dS_L=7 << 45, dq=8 << 45, dk_=9 << 45, dv_=10 << 45,
          dlog_a=11 << 45, dS0=12 << 45, ws=13 << 45), UNSUPPORTED),
])
def test_gated_bwd_chunk(lib, over, status):
    assert _call(lib.falcon_gated_bwd_chunk, BWD, over) == status


def test_gated_workspaces(lib):
    f, b = lib.falcon_gated_fwd_workspace_bytes, lib.falcon_gated_bwd_workspace_bytes
    assert f(1, 1, 64, 64, 64, 0) == 0               # one chunk
    assert f(64, 16, 8192, 64, 64, 0) == 0           # chains enough to fill the GPU
    assert f(1, 4, 32768, 128, 128, 0) > 0
    assert f(1, 1, 0, 64, 64, 0) == b(1, 1, 64, 48, 64, 0) == b(1, 1, 64, 64, 64, 3) == 0
    assert b(1, 1, 1, 16, 16, 0) > 0
