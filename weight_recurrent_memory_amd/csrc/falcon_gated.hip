// falcon_gated.hip - forward of the gated linear recurrence over a sequence:
//   S_t = a_t S_{t-1} + v_t k_t^T,   o_t = S_t q_t,   a = exp(log_a)
// by the chunk kernel of falcon_gated_chunk.h.  A long sequence of few chains is cut into
// segments until some 768 workgroups run: a first kernel forms each segment's own write to
// the state from zero (k and v only), a second runs the short recurrence over segments,
// and the main kernel starts each segment from its state.
#include "falcon_gated_chunk.h"

namespace falcon {
namespace gated {

// The recurrence over segments: start of step j + 1 = decay_j start_j + write_j, in place,
// slot 0 set to U0 (so that the last segment may write its result over U0).
__global__ __launch_bounds__(256) void segments_kernel(const float* U0, Span sp, long size4) {
  const long per = (size4 + 255) / 256;
  const long chain = blockIdx.x / per, i = (blockIdx.x % per) * 256 + threadIdx.x;
  if (i >= size4) return;
  float4* s = reinterpret_cast<float4*>(sp.states) + chain * (sp.writes + 1) * size4 + i;
  const float* d = sp.decays + chain * sp.writes;
  float4 x = {0.f, 0.f, 0.f, 0.f};
  if (U0) x = reinterpret_cast<const float4*>(U0)[chain * size4 + i];
  *s = x;
  s += size4;
  for (int j0 = 0; j0 < sp.writes; j0 += 8) {
    float4 w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j0 + j < sp.writes) w[j] = s[(j0 + j) * size4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j0 + j < sp.writes) {
        const float a = d[j0 + j];
        x = float4{a * x.x + w[j].x, a * x.y + w[j].y, a * x.z + w[j].z, a * x.w + w[j].w};
        s[(j0 + j) * size4] = x;
      }
    }
  }
}

hipError_t launch_segments(const float* U0, const Span& sp, long chains, long state, hipStream_t stream) {
  const long size4 = state / 4;
  hipLaunchKernelGGL(segments_kernel, dim3((unsigned)(chains * ((size4 + 255) / 256))), dim3(256), 0,
                     stream, U0, sp, size4);
  return hipGetLastError();
}

namespace {

// One workgroup's walk takes any number of chunks.
Span cut_of(const GatedArgs& a) {
  const long blocks = a.dv / rows_of(a.dv);
  Span sp = cut((long)a.batch * a.heads * blocks, a.seqlen, 1l << 40);
  sp.writes = sp.segs - 1;
  return sp;
}

template <typename T>
hipError_t run(const GatedArgs& a, const Span& sp, hipStream_t stream) {
  const ChunkArgs c{a.k, a.q, a.v, a.log_a, a.S0, a.o, a.S_out, nullptr, nullptr,
                    (long)a.batch * a.heads, a.seqlen, a.dv};
  const hipError_t e = launch_states<T, T, false>(c, a.dk, sp, stream);
  if (e != hipSuccess) return e;
  return with_sizes(a.dk, a.dv, [&](auto d, auto r) {
    return go_chunk<T, T, T, decltype(d)::value, decltype(r)::value, false, false>(c, sp, stream);
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
    sp = gated::Span{1, (a.seqlen + gated::C - 1) / gated::C, 0, nullptr, nullptr};
  }
  return a.dtype == 0 ? gated::run<uint16_t>(a, sp, stream) : gated::run<float>(a, sp, stream);
}

}  // namespace falcon
