// falcon_delta.h - shared pieces of the gated delta rule's chunk kernels.
//
//   S_t = a_t S_{t-1} + u_t k_t^T,  u_t = b_t (v_t - a_t S_{t-1} k_t),  o_t = S_t q_t
// In a chunk of 64 tokens, with S the state before it, D_ts the decay from s to t, e_t from
// the chunk's start to t, w_s from s to its end and d the whole chunk's:
//   A_ts = b_t D_ts (k_t . k_s) for s < t,  T = (I + A)^-1
//   X = b (V - e (K S^T)),  U = T X,  S <- d S + sum_s w_s u_s k_s^T
//   o_t = e_t S q_t + sum_{s<=t} D_ts (q_t . k_s) u_s
// T needs keys and gates only and is formed for all chunks side by side; what is left in
// order is S -> X -> U -> S.
//
// The walk in order holds S^T (columns of keys by value rows) in accumulators and needs no
// exchange between lanes: a 16x16 product's result has row 4 g + r and column m on lane
// (m = lane % 16, g = lane / 16), and an operand's lane m has 8 slots of its column, so two
// results of tiles 2 j and 2 j + 1 are one operand whose slots mean rows 32 j + 4 g + 0..3
// and 32 j + 16 + 4 g + 0..3.  Every other operand here is read in this order of slots
// ("paired order").  The planes, decays and windows are falcon_gated.h's.
#pragma once
#include <type_traits>

#include "falcon_block_launch.h"
#include "falcon_gated.h"

namespace falcon {
namespace delta {

using namespace gated;      // C, planes, split3, frag3, Window, Raw4, decays

// Orders a wave's own LDS traffic.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The wave of a workgroup, as a scalar: what goes by it needs no lane masks.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); }

// T as operands of rows t, in paired order of s: of row tile i the 32-token steps 0..i/2.
constexpr int kFrags = 6;
__host__ __device__ constexpr int frag_of(int i, int j) { return i < 2 ? i : 2 * i - 2 + j; }
constexpr int kT = kFrags * 3 * 64;          // uint4 of a chunk's T

// Operand planes of two result tiles (or none in the second's place).
__device__ __forceinline__ void frag_pair(const floatx4& a, const floatx4& b, bf16x8 (&f)[3]) {
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  frag3(x, f);
}

// One row in paired order on its way from memory: columns 32 i + 4 g .. and 32 i + 16 + 4 g ..
template <typename T, int D>
struct PairRow {
  static constexpr int NP = planes<T>(), N = (D + 31) / 32;
  Raw4<T> lo[N], hi[N];
  // row: of the window's
  __device__ __forceinline__ void load(const Window& w, int row) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      lo[i].load(w, (row * D + 32 * i + 4 * g) * (int)sizeof(T));
      hi[i].load(w, 32 * i + 16 < D ? (row * D + 32 * i + 16 + 4 * g) * (int)sizeof(T) : kNowhere);
    }
  }
  __device__ __forceinline__ void frag(int i, bf16x8 (&f)[NP]) const {
    if constexpr (NP == 1) {
      f[0] = __builtin_bit_cast(bf16x8, uint4{lo[i].u.x, lo[i].u.y, hi[i].u.x, hi[i].u.y});
    } else {
      frag_pair(lo[i].values(), hi[i].values(), f);
    }
  }
};

// The same from planes in LDS, rows of D.
template <int NP, int D>
__device__ __forceinline__ void pair_frag(const uint16_t* p, int row, int i, bf16x8 (&f)[NP]) {
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    const uint2 lo = *reinterpret_cast<const uint2*>(p + n * C * D + at<D>(row, 32 * i + 4 * g));
    uint2 hi = {0u, 0u};
    if (32 * i + 16 < D) hi = *reinterpret_cast<const uint2*>(p + n * C * D + at<D>(row, 32 * i + 16 + 4 * g));
    f[n] = __builtin_bit_cast(bf16x8, uint4{lo.x, lo.y, hi.x, hi.y});
  }
}

// Columns 16 j .. of the transposed planes, tokens 32 kk .. in paired order.
template <int NP, int D>
__device__ __forceinline__ void pair_frag_t(const uint16_t* p, int kk, int j, bf16x8 (&f)[NP]) {
  typedef __attribute__((address_space(3))) short4_t* lds_ptr;
  const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  const int row = 32 * kk + 4 * g + (m >> 2), col = 16 * j + 4 * (m & 3);
  const int a = at<D>(row, col), b = at<D>(row + 16, col);
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    struct { short4_t lo, hi; } x;
    x.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + n * C * D + a));
    x.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + n * C * D + b));
    f[n] = __builtin_bit_cast(bf16x8, x);
  }
}

// A float of a window at `at` bytes.
__device__ __forceinline__ float load_f32(const Window& w, int at) {
  return __builtin_bit_cast(float, w.load4b(at));
}
// One input of a window at element i.
__device__ __forceinline__ float load_one(const Window& w, int i, uint16_t) {
  return bf16_to_f32((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(w.r, 2 * i, 0, 0));
}
__device__ __forceinline__ float load_one(const Window& w, int i, float) { return load_f32(w, 4 * i); }

// Four consecutive floats in LDS, 16-byte aligned.
__device__ __forceinline__ floatx4 four(const float* p) {
  return *static_cast<const floatx4*>(__builtin_assume_aligned(p, 16));
}

// A chunk's gates, one token a lane.
struct Gates {
  alignas(16) float2 g[C];           // sums of log2 decays
  alignas(16) float e[C];
  alignas(16) float w[C];
  alignas(16) float b[C];
  alignas(16) float be[C];
  float d;
};
struct GateLoad {
  float raw, beta;
  __device__ __forceinline__ void load(const float* log_a, const float* b, long t0, long len) {
    const int at = 4 * (threadIdx.x & 63);
    raw = load_f32(Window(log_a ? log_a + t0 : b, log_a ? len - t0 : 0, 1, 0), at);
    beta = load_f32(Window(b + t0, len - t0, 1, 0), at);
  }
  __device__ __forceinline__ void store(Gates& x) const {
    const int lane = threadIdx.x & 63;
    const double s = wave_scan(log2_decay(raw)), all = __shfl(s, 63, 64);
    const float e = exp2_of(s);
    x.g[lane] = two_floats(s);
    x.e[lane] = e;
    x.w[lane] = exp2_of(all - s);
    x.b[lane] = beta;
    x.be[lane] = beta * e;
    if (lane == 0) x.d = exp2_of(all);
  }
};

// A kernel with more than 64 KB of LDS has to be told so.
template <class K>
hipError_t lds_limit(K kernel, size_t bytes) {
  if (bytes <= 65536) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// f(size) as a constant.
template <class F>
hipError_t with_dim(int d, F&& f) {
  switch (d) {
    case 16: return f(std::integral_constant<int, 16>());
    case 32: return f(std::integral_constant<int, 32>());
    case 64: return f(std::integral_constant<int, 64>());
    case 128: return f(std::integral_constant<int, 128>());
  }
  return hipErrorInvalidValue;
}

// Whether a launch of grid_of(blocks, units) workgroups has fewer than 2^32 work-items.
inline bool fits(long blocks, long units, long threads) {
  return (units + 7) / 8 * 8 * blocks * threads < (1l << 32);
}

struct SolveArgs {
  const void* k;             // [chain][L][dk]
  const float* beta;         // [chain][L]
  const float* log_a;        // [chain][L], or null
  uint4* T;                  // [chain][chunk][kT]
  uint4* Tt;                 // the transposed, or null
  long chains;
  int seqlen;
};
// Every chunk's T (falcon_delta_solve.hip), four chunks a workgroup of 256.
constexpr int kSolveWaves = 4;
inline bool solve_fits(long chunks) { return (chunks + kSolveWaves - 1) / kSolveWaves * 64 * kSolveWaves < (1l << 32); }
hipError_t launch_solve(const SolveArgs& a, int dk, int dtype, hipStream_t stream);

}  // namespace delta
}  // namespace falcon
