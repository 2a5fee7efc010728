// falcon_gated_bwd.hip - gradients of the gated linear recurrence.
//
// With R_t the gradient of S_t (R_L = dS_L + dO_L q_L^T, R_t = a_{t+1} R_{t+1} + dO_t q_t^T):
//   dq_t = S_t^T dO_t,   dk_t = R_t^T v_t,   dv_t = R_t k_t,   dS0 = a_1 R_1
//   dlog_a_t = a_t <R_t, S_{t-1}>
// dq, dk and dv have the forward's own form (falcon_gated_chunk.h), dk and dv last token
// first.  dlog_a_t is the part of the loss that passes the border between t - 1 and t: over
// all writes s (S0 among them) and reads t' (dS_L among them) the sum of their products
// with s < t <= t'.  The dq kernel gives r_t' = q_t' . dq_t', the dk kernel c_s = k_s . dk_s,
// both without the product of a token with itself, which passes no border and would only
// leave its rounding behind; then inside a segment
//   dlog_a_t = X + sum_{t'>=t} r_t' - sum_{s>=t} c_s,   X = <R, S> at the segment's end,
// summed in float64.  Segments are 16 chunks at most, so that an X is never far away.
#include "falcon_gated_chunk.h"

namespace falcon {
namespace gated {
namespace {

constexpr int kMostChunks = 16;            // of a segment: 1024 tokens

struct GateArgs {
  const float* log_a;
  const float* dS_L;       // or null
  const float* r;          // [block][chain][L]
  const float* c;
  int blocks;
  float* dlog_a;
  long chains, state;
  int seqlen;
};

__device__ __forceinline__ double block_sum(double x, double* lds) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  return lds[0] + lds[1] + lds[2] + lds[3];
}

// One segment of one chain: four tokens a thread.
__global__ __launch_bounds__(NT) void gate_kernel(GateArgs a, Span s, Span r) {
  __shared__ double lds[4];
  const long chain = blockIdx.x / s.segs;
  const int seg = (int)(blockIdx.x % s.segs);
  const bool last = seg == s.segs - 1;
  const float* R = last ? a.dS_L : r.states;
  double x = 0.0;
  if (R) {
    R += last ? chain * a.state : (chain * (r.writes + 1) + s.segs - 1 - seg) * a.state;
    const float* S = s.states + (chain * (s.writes + 1) + seg + 1) * a.state;
    for (long i = threadIdx.x * 4; i < a.state; i += NT * 4) {
      const float4 p = *reinterpret_cast<const float4*>(R + i), q = *reinterpret_cast<const float4*>(S + i);
      x += (double)p.x * q.x + (double)p.y * q.y + (double)p.z * q.z + (double)p.w * q.w;
    }
  }
  const double X = block_sum(x, lds);
  const long len = a.seqlen, t0 = (long)seg * s.chunks * C;
  const long end = t0 + (long)s.chunks * C < len ? t0 + (long)s.chunks * C : len;
  // thread i: the four tokens 4 i .. from the segment's last one backward
  double sum[4], mine = 0.0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long t = end - 1 - 4 * (long)threadIdx.x - j;
    double rr = 0.0, cc = 0.0;
    if (t >= t0) {
      for (int b = 0; b < a.blocks; ++b) {
        rr += a.r[(b * a.chains + chain) * len + t];
        cc += a.c[(b * a.chains + chain) * len + t];
      }
    }
    mine += rr - cc;
    sum[j] = mine;
  }
  const double upto = wave_scan(mine);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = upto;
  __syncthreads();
  double before = X + upto - mine;
  for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) before += lds[w];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long t = end - 1 - 4 * (long)threadIdx.x - j;
    // nothing passes a reset
    if (t >= t0) a.dlog_a[chain * len + t] = a.log_a[chain * len + t] < -1000.0f ? 0.0f : (float)(before + sum[j]);
  }
}

// Both directions' states, and all three gradients, in one launch each: the workgroups
// of one chain's segment run near each other in time and share its rows in the L2, and
// one launch's last workgroups leave no part of the GPU idle.  (Up to 64 columns; at 128
// the largest of the LDS needs, dk's 104 KB, would hold the others to one workgroup a
// compute unit.)
template <typename T, int DK, int DV>
__global__ __launch_bounds__(NT) void both_states_kernel(ChunkArgs S, Span s, ChunkArgs R, Span r) {
  extern __shared__ __align__(16) unsigned char smem[];
  int blk;
  long unit;
  const long ns = S.chains * s.writes, nr = R.chains * r.writes;
  if (!place(2, ns > nr ? ns : nr, blk, unit)) return;
  if (blk == 0) {
    if (unit < ns) state_body<T, T, DK, DV, false>(S, s, 0, unit, smem);
  } else {
    if (unit < nr) state_body<T, float, DK, DV, true>(R, r, 0, unit, smem);
  }
}
template <typename T, int DK, int DV>
__global__ __launch_bounds__(NT, 2) void gradients_kernel(ChunkArgs q, ChunkArgs k, ChunkArgs v, Span s, Span r) {
  extern __shared__ __align__(16) unsigned char smem[];
  int blk;
  long unit;
  if (!place(3, q.chains * s.segs, blk, unit)) return;
  if (blk == 0) chunk_body<float, T, T, DV, DK, true, true>(k, r, 0, unit, smem);
  else if (blk == 1) chunk_body<T, float, T, DV, DK, false, true>(q, s, 0, unit, smem);
  else chunk_body<T, T, float, DK, DV, true, false>(v, r, 0, unit, smem);
}
template <typename T, int DK, int DV>
hipError_t both(const ChunkArgs& S, const ChunkArgs& R, const ChunkArgs& q, const ChunkArgs& k,
                const ChunkArgs& v, const Span& s, const Span& r, hipStream_t stream) {
  hipError_t e;
  const long writes = s.writes > r.writes ? s.writes : r.writes;
  if (writes > 0) {
    constexpr size_t bytes = sizeof(LdsState<T, float, DK, DV>);
    auto kernel = both_states_kernel<T, DK, DV>;
    if ((e = lds_limit(kernel, bytes)) != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(grid_of(2, S.chains * writes)), dim3(NT), bytes, stream, S, s, R, r);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if ((e = launch_segments(S.U0, s, R.U0, r, S.chains, (long)DK * DV, stream)) != hipSuccess) return e;
  }
  constexpr size_t a = sizeof(Lds<float, T, DV, DK>), b = sizeof(Lds<T, float, DK, DV>);
  constexpr size_t bytes = a > b ? a : b;
  auto kernel = gradients_kernel<T, DK, DV>;
  if ((e = lds_limit(kernel, bytes)) != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(grid_of(3, S.chains * s.segs)), dim3(NT), bytes, stream, q, k, v, s, r);
  return hipGetLastError();
}
// f(dk, dv) as constants up to 64
template <class F>
hipError_t with_small(int dk, int dv, F&& f) {
  auto cols = [&](auto k) {
    switch (dv) {
      case 16: return f(k, std::integral_constant<int, 16>());
      case 32: return f(k, std::integral_constant<int, 32>());
      case 64: return f(k, std::integral_constant<int, 64>());
    }
    return hipErrorInvalidValue;
  };
  switch (dk) {
    case 16: return cols(std::integral_constant<int, 16>());
    case 32: return cols(std::integral_constant<int, 32>());
    case 64: return cols(std::integral_constant<int, 64>());
  }
  return hipErrorInvalidValue;
}

// The two spans of a call (states first token first, their gradients last token first)
// and its workspace.
struct Plan {
  Span s, r;
  int blocks;              // of dq's and dk's columns
  long chains, state;
  size_t bytes() const {
    return span_bytes(s, chains, state) + span_bytes(r, chains, state);
  }
};

Plan plan_of(const GatedBwdArgs& a) {
  Plan p;
  p.chains = (long)a.batch * a.heads;
  p.state = (long)a.ndv * a.ndk;
  p.blocks = a.ndk / rows_of(a.ndk);
  p.s = cut(p.chains * p.blocks, a.seqlen, kMostChunks);
  p.r = p.s;
  // the end's state only where its gradient meets it
  p.s.writes = a.dS_L && a.dlog_a ? p.s.segs : p.s.segs - 1;
  p.r.writes = p.r.segs - 1;
  return p;
}
size_t dot_floats(const Plan& p, const GatedBwdArgs& a) {
  return a.dlog_a ? (size_t)2 * p.blocks * p.chains * a.seqlen : 0;
}

template <typename T>
hipError_t run(const GatedBwdArgs& a, Plan p, hipStream_t stream) {
  float* w = a.workspace;
  place_span(p.s, p.chains, p.state, w);
  place_span(p.r, p.chains, p.state, w);
  float* r = a.dlog_a ? w : nullptr;
  float* c = a.dlog_a ? w + (size_t)p.blocks * p.chains * a.seqlen : nullptr;
  hipError_t e;
  const ChunkArgs S{a.k, nullptr, a.v, a.log_a, a.S0, nullptr, nullptr, nullptr, nullptr, p.chains, a.seqlen, a.ndv};
  const ChunkArgs R{a.q, nullptr, a.dO, a.log_a, a.dS_L, nullptr, nullptr, nullptr, nullptr, p.chains, a.seqlen, a.ndv};
  const ChunkArgs dq{a.v, a.dO, a.k, a.log_a, a.S0, a.dq, nullptr, a.q, r, p.chains, a.seqlen, a.ndk};
  const ChunkArgs dk{a.dO, a.v, a.q, a.log_a, a.dS_L, a.dk, nullptr, a.k, c, p.chains, a.seqlen, a.ndk};
  const ChunkArgs dv{a.q, a.k, a.dO, a.log_a, a.dS_L, a.dv, a.dS0, nullptr, nullptr, p.chains, a.seqlen, a.ndv};
  if (a.ndk <= 64 && a.ndv <= 64) {
    e = with_small(a.ndk, a.ndv, [&](auto nk, auto nv) {
      return both<T, decltype(nk)::value, decltype(nv)::value>(S, R, dq, dk, dv, p.s, p.r, stream);
    });
  } else {
    if ((e = launch_states<T, T, false>(S, a.ndk, p.s, stream)) != hipSuccess) return e;
    if ((e = launch_states<T, float, true>(R, a.ndk, p.r, stream)) != hipSuccess) return e;
    e = with_sizes(a.ndv, a.ndk, [&](auto d, auto z) {
      return go_chunk<T, float, T, decltype(d)::value, decltype(z)::value, false, true>(dq, p.s, stream);
    });
    if (e != hipSuccess) return e;
    e = with_sizes(a.ndv, a.ndk, [&](auto d, auto z) {
      return go_chunk<float, T, T, decltype(d)::value, decltype(z)::value, true, true>(dk, p.r, stream);
    });
    if (e != hipSuccess) return e;
    e = with_sizes(a.ndk, a.ndv, [&](auto d, auto z) {
      return go_chunk<T, T, float, decltype(d)::value, decltype(z)::value, true, false>(dv, p.r, stream);
    });
  }
  if (e != hipSuccess || !a.dlog_a) return e;
  const GateArgs g{a.log_a, a.dS_L, r, c, p.blocks, a.dlog_a, p.chains, p.state, a.seqlen};
  hipLaunchKernelGGL(gate_kernel, dim3((unsigned)(p.chains * p.s.segs)), dim3(NT), 0, stream, g, p.s, p.r);
  return hipGetLastError();
}

}  // namespace
}  // namespace gated

size_t gated_bwd_workspace_bytes(const GatedBwdArgs& a) {
  const gated::Plan p = gated::plan_of(a);
  return p.bytes() + gated::dot_floats(p, a) * sizeof(float);
}

hipError_t launch_gated_bwd(const GatedBwdArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  const gated::Plan p = gated::plan_of(a);
  return a.dtype == 0 ? gated::run<uint16_t>(a, p, stream) : gated::run<float>(a, p, stream);
}

}  // namespace falcon
