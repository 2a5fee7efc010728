// falcon_gated.hip - forward of the gated linear recurrence over a sequence:
//   S_t = a_t S_{t-1} + v_t k_t^T,   o_t = S_t q_t,   a = exp(log_a)
// by the chunk kernel of falcon_gated_chunk.h.  A long sequence of few chains is cut into
// segments until some 768 workgroups run: a first kernel forms each segment's own write to
// the state from zero (k and v only), a second runs the short recurrence over segments,
// and the main kernel starts each segment from its state.  8x12x2048x64 bf16: 14 + 8 + 30 us
// in three kernels, 46-52 us a call (walked whole, on 96 workgroups, 77 us); 1x4x32771x128:
// 26 + 9 + 60 us, 84-91 us a call (walked whole 1664 us).
#include "falcon_gated_chunk.h"

namespace falcon {
namespace gated {
namespace {

// The recurrence over segments: start of step j + 1 = decay_j start_j + write_j, in place,
// slot 0 set to U0 (so that the last segment may write its result over U0).  Of one span
// (blockIdx.y 0) or two.
__global__ __launch_bounds__(256) void segments_kernel(const float* U0, Span sp, const float* U1, Span sp1,
                                                       long size) {
  if (blockIdx.y) {
    U0 = U1;
    sp = sp1;
  }
  if (sp.writes == 0) return;
  const long per = size / 256;               // size is a multiple of 256
  const long chain = blockIdx.x / per, i = (blockIdx.x % per) * 256 + threadIdx.x;
  float* s = sp.states + chain * (sp.writes + 1) * size + i;
  const float* d = sp.decays + chain * sp.writes;
  float x = U0 ? U0[chain * size + i] : 0.0f;
  *s = x;
  s += size;
  constexpr int N = 16;                      // loads in flight
  for (int j0 = 0; j0 < sp.writes; j0 += N) {
    float w[N], a[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const bool in = j0 + j < sp.writes;
      w[j] = in ? s[(j0 + j) * size] : 0.0f;
      a[j] = in ? d[j0 + j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j0 + j < sp.writes) {
        x = a[j] * x + w[j];
        s[(j0 + j) * size] = x;
      }
    }
  }
}

}  // namespace

hipError_t launch_segments(const float* U0, const Span& sp, const float* U1, const Span& sp1, long chains,
                           long state, hipStream_t stream) {
  hipLaunchKernelGGL(segments_kernel, dim3((unsigned)(chains * (state / 256)), sp1.writes ? 2 : 1),
                     dim3(256), 0, stream, U0, sp, U1, sp1, state);
  return hipGetLastError();
}

namespace {

// One workgroup's walk takes any number of chunks.  256 compute units hold two or three
// workgroups of the chunk kernel each, one with float32 inputs at 128 columns.
constexpr long kWhole = 13;
int block_of(const GatedArgs& a) { return rows_of(a.dv, (long)a.batch * a.heads, a.seqlen, kWhole); }
Span cut_of(const GatedArgs& a) {
  const long blocks = a.dv / block_of(a);
  const long held = a.dtype == 0 ? (a.dk <= 64 ? 3 : 2) : (a.dk <= 64 ? 2 : 1);
  Span sp = cut((long)a.batch * a.heads * blocks, a.seqlen, 256 * held, 1l << 40, kWhole);
  sp.writes = sp.segs - 1;
  return sp;
}

template <typename T>
hipError_t run(const GatedArgs& a, const Span& sp, hipStream_t stream) {
  const ChunkArgs c{a.k, a.q, a.v, a.log_a, a.S0, a.o, a.S_out, nullptr, nullptr,
                    (long)a.batch * a.heads, a.seqlen, a.dv};
  const hipError_t e = launch_states<T, T, false>(c, a.dk, block_of(a), sp, stream);
  if (e != hipSuccess) return e;
  return with_sizes(a.dk, block_of(a), [&](auto d, auto r) {
    return go_chunk<T, decltype(d)::value, decltype(r)::value>(c, sp, stream);
  });
}

}  // namespace
}  // namespace gated

size_t gated_workspace_bytes(const GatedArgs& a) {
  return gated::span_bytes(gated::cut_of(a), (long)a.batch * a.heads, (long)a.dv * a.dk);
}

hipError_t launch_gated(const GatedArgs& a, void* ws, size_t ws_bytes, hipStream_t stream) {
  (void)hipGetLastError();
  gated::Span sp = gated::cut_of(a);
  if (ws && ws_bytes >= gated_workspace_bytes(a)) {
    float* p = static_cast<float*>(ws);
    gated::place_span(sp, (long)a.batch * a.heads, (long)a.dv * a.dk, p);
  } else {
    sp = gated::Span{1, (int)(((long)a.seqlen + gated::C - 1) / gated::C), 0, nullptr, nullptr};
  }
  return a.dtype == 0 ? gated::run<uint16_t>(a, sp, stream) : gated::run<float>(a, sp, stream);
}

}  // namespace falcon
