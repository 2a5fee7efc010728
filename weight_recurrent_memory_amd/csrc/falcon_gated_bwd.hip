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
// summed in float64.  Segments are 16 chunks at most, so that an X is never far away; at
// a reset, any token whose float32 decay is 0, the sum is 0 and begins anew: no product
// passes it, and the rounding left by one document's sums stays out of another's.
//
// Four launches: both directions' segment writes, their recurrences, the three gradients,
// the gates.  8x12x2048x64 bf16: 30 + 13 + 109 + 8 us (131-152 us a call from GPU to GPU, the
// kernels partly overlapping); the gradients move 422 MB over the fabric (inputs read by
// the dk and dv part and again by the dq part, 3.9 TB/s) and issue 540 vector and 86
// matrix instructions a chunk and wave on two waves a SIMD: bound by both.  Tried: three parts in
// place of two (157 us), blocks of 32 columns (180 us), segments of two chunks for this
// shape (179 us), each part a launch of its own (188 us).
#include "falcon_gated_chunk.h"

namespace falcon {
namespace gated {
namespace {

constexpr int kMostChunks = 16;            // of a segment: 1024 tokens
// Chunks from which a sequence is cut: where few workgroups would walk it whole (us cut and
// whole: 1x8x512x64 29 and 48), at 128 columns (1x3x320x128: 37 and 28), where 192 do
// (8x12x512x64 58 and 49, 2x8x512x128 52 and 43) and where 320 do (16x12x1000x64: 142 and
// 107; a whole segment's chunks).
constexpr long kWholeFew = 5, kWholeWide = 8, kWholeMany = 13, kMany = 192, kMost = 320;

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
  // thread i: the four tokens 4 i .. from the segment's last one backward; `cut` once a
  // reset has begun the sum anew
  double sum[4], mine = 0.0;
  bool cut = false, reset[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long t = end - 1 - 4 * (long)threadIdx.x - j;
    double rr = 0.0, cc = 0.0;
    reset[j] = false;
    if (t >= t0) {
      for (int b = 0; b < a.blocks; ++b) {
        rr += a.r[(b * a.chains + chain) * len + t];
        cc += a.c[(b * a.chains + chain) * len + t];
      }
      reset[j] = is_reset(a.log_a[chain * len + t]);
    }
    mine += rr - cc;
    sum[j] = mine;
    if (reset[j]) {
      mine = 0.0;
      cut = true;
    }
  }
  // the sum, and whether a reset lies in it, up to and with each thread, then before it
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double upto = mine;
  int any = cut;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double y = __shfl_up(upto, m, 64);
    const int f = __shfl_up(any, m, 64);
    if (lane >= m) {
      if (!any) upto += y;
      any |= f;
    }
  }
  __syncthreads();
  __shared__ int flag[4];
  if (lane == 63) {
    lds[wave] = upto;
    flag[wave] = any;
  }
  __syncthreads();
  double before = X;
  for (int w = 0; w < wave; ++w) before = flag[w] ? lds[w] : before + lds[w];
  const double up = __shfl_up(upto, 1, 64);
  const int upf = __shfl_up(any, 1, 64);
  if (lane > 0) before = upf ? up : before + up;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long t = end - 1 - 4 * (long)threadIdx.x - j;
    if (t >= t0) a.dlog_a[chain * len + t] = reset[j] ? 0.0f : (float)(before + sum[j]);
    if (reset[j]) before = 0.0;
  }
}

// dk and dv together, up to 64 columns each, last token first: one R for both, read by
// rows for dv and transposed for dk, and one place in LDS for q and dO, which are x and z
// of the one and z and x of the other.
template <typename T, int DK, int DV>
struct LdsKV {
  static constexpr int NPX = planes<T>(), NPZ = 3;
  static constexpr int W = DK < 32 ? 32 : DK, WZ = DV < 32 ? 32 : DV;   // k-slots in 32s
  alignas(16) uint16_t x[NPX][C * W];               // q
  alignas(16) uint16_t z[NPZ][C * WZ];              // dO
  alignas(16) uint16_t s[3][WZ * W];                // R at the chunk's start
  alignas(16) float2 g[C];
  alignas(16) float e[C];
  alignas(16) float w[C];
  float d;
};

struct KVArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* dO;
  const float* log_a;
  const float* dS_L;
  float* dk;
  float* dv;
  float* dS0;
  float* dots;             // or null
  long chains;
  int seqlen;
};

template <typename T, int DK, int DV>
__device__ __forceinline__ void kv_body(const KVArgs& a, const Span& sp, long unit, unsigned char* smem) {
  using L = LdsKV<T, DK, DV>;
  constexpr int NP = L::NPX, W = L::W, WZ = L::WZ, NK = W / 32, NV = WZ / 32, TK = DK / 16, TV = DV / 16;
  L& lds = *reinterpret_cast<L*>(smem);
  const long chain = unit / sp.segs, len = a.seqlen;
  const int step = (int)(unit % sp.segs);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const Walk<true> walk(sp, step, len);
  const T* q = static_cast<const T*>(a.q) + chain * len * DK;
  const T* k = static_cast<const T*>(a.k) + chain * len * DK;
  const T* v = static_cast<const T*>(a.v) + chain * len * DV;
  const float* dO = a.dO + chain * len * DV;
  const float* la = a.log_a ? a.log_a + chain * len : nullptr;
  float* dk = a.dk + chain * len * DK;
  float* dv = a.dv + chain * len * DV;
  constexpr long state = (long)DV * DK;
  const int ti = 16 * wave + m;

  Stage<T, DK, true> sx(DK);
  Stage<float, DV, true> sz(DV);
  State<DK, DV> st;
  Decays dec;
  Row<T, DK, true> rk;
  Row<T, DV, true> rv;
  const int u_at = (row_at<true>(ti) * DK + 4 * g) * (int)sizeof(T);
  auto fetch = [&](long t0) {
    sx.load(Window(q + t0 * DK, len - t0, DK, 0));
    sz.load(Window(dO + t0 * DV, len - t0, DV, 0));
    rk.load(Window(k + t0 * DK, len - t0, DK, 0));
    rv.load(Window(v + t0 * DV, len - t0, DV, 0));
  };
  dec.load<true>(la, walk.at(0), len);
  fetch(walk.at(0));
  dec.sum<true>();
  if (walk.n > 1) dec.load<true>(la, walk.at(1), len);
  if (sp.segs > 1) st.load(sp.states + (chain * (sp.writes + 1) + step) * state, DK, 1);
  else st.load(a.dS_L ? a.dS_L + chain * state : nullptr, DK, 1);
  if (DK < W || DV < WZ) {
    for (int i = threadIdx.x; i < NP * C * W / 8; i += NT) reinterpret_cast<uint4*>(lds.x[0])[i] = uint4{0u, 0u, 0u, 0u};
    for (int i = threadIdx.x; i < 3 * C * WZ / 8; i += NT) reinterpret_cast<uint4*>(lds.z[0])[i] = uint4{0u, 0u, 0u, 0u};
    for (int i = threadIdx.x; i < 3 * WZ * W / 8; i += NT) reinterpret_cast<uint4*>(lds.s[0])[i] = uint4{0u, 0u, 0u, 0u};
    __syncthreads();
  }

  for (int c = 0; c < walk.n; ++c) {
    if (c) __syncthreads();
    sx.template store<W>(lds.x[0]);
    sz.template store<WZ>(lds.z[0]);
    st.template to_planes<W>(lds.s[0], WZ * W);
    if (wave == 0) dec.store(lds);
    bf16x8 kf[NK][NP], vf[NV][NP];
    rk.frags(kf);
    rv.frags(vf);
    __syncthreads();
    const long t = token<true>(walk.at(c), ti);
    Raw4<T> ru[TK];        // k again, as dk's columns lie on the lanes
    const Window wk(k + walk.at(c) * DK, len - walk.at(c), DK, 0);
#pragma unroll
    for (int d = 0; d < TK; ++d) ru[d].load(wk, u_at + 16 * d * (int)sizeof(T));
    if (wave == 0) dec.sum<true>();
    if (c + 2 < walk.n) dec.load<true>(la, walk.at(c + 2), len);
    if (c + 1 < walk.n) fetch(walk.at(c + 1));

    // the part of what lies behind the chunk: e R k and e R^T v
    floatx4 av[TV], ak[TK];
#pragma unroll
    for (int d = 0; d < TV; ++d) av[d] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int d = 0; d < TK; ++d) ak[d] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      bf16x8 s[TV][3];
#pragma unroll
      for (int d = 0; d < TV; ++d) frag<3, W>(lds.s[0], WZ * W, 16 * d + m, 32 * i + 8 * g, s[d]);
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int r = 0; r < NP; ++r)
          if (p + r < 3) {
#pragma unroll
            for (int d = 0; d < TV; ++d) av[d] = mfma16(s[d][p], kf[i][r], av[d]);
          }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      bf16x8 s[TK][3];
#pragma unroll
      for (int d = 0; d < TK; ++d) frag_t<3, W>(lds.s[0], WZ * W, 32 * i + 8 * g, 16 * d, s[d]);
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int r = 0; r < NP; ++r)
          if (p + r < 3) {
#pragma unroll
            for (int d = 0; d < TK; ++d) ak[d] = mfma16(s[d][p], vf[i][r], ak[d]);
          }
    }
    const float e = lds.e[ti];
    const float2 Gt = lds.g[ti];
#pragma unroll
    for (int d = 0; d < TV; ++d) av[d] *= e;
#pragma unroll
    for (int d = 0; d < TK; ++d) ak[d] *= e;
    float same = 0.0f;     // v_t . dO_t, where this lane holds it
#pragma unroll
    for (int kk = 0; kk < C; kk += 32) {
      if (kk > 16 * wave + 15) break;
      __builtin_amdgcn_sched_barrier(0);
      float x[8], y[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = kk + 8 * (m >> 2) + 4 * j + (m & 3);
        floatx4 pq = {0.f, 0.f, 0.f, 0.f}, pv = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          bf16x8 f[NP];
          frag<NP, W>(lds.x[0], C * W, row, 32 * i + 8 * g, f);
          mma<NP, NP>(f, kf[i], pq);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          bf16x8 f[3];
          frag<3, WZ>(lds.z[0], C * WZ, row, 32 * i + 8 * g, f);
          mma<3, NP>(f, vf[i], pv);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int s = kk + 8 * g + 4 * j + r;
          const float dcy = decay(Gt, lds.g[s]);
          x[4 * j + r] = s <= ti ? pq[r] * dcy : 0.0f;
          y[4 * j + r] = s < ti ? pv[r] * dcy : 0.0f;
          same = s == ti ? pv[r] : same;
        }
      }
      bf16x8 pf[3];
      frag3(x, pf);
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        bf16x8 f[TV][1];
#pragma unroll
        for (int d = 0; d < TV; ++d) frag_t<1, WZ>(lds.z[p], 0, kk + 8 * g, 16 * d, f[d]);
#pragma unroll
        for (int r = 0; p + r < 3; ++r)
#pragma unroll
          for (int d = 0; d < TV; ++d) av[d] = mfma16(f[d][0], pf[r], av[d]);
      }
      __builtin_amdgcn_sched_barrier(0);
      frag3(y, pf);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        bf16x8 f[TK][1];
#pragma unroll
        for (int d = 0; d < TK; ++d) frag_t<1, W>(lds.x[p], 0, kk + 8 * g, 16 * d, f[d]);
#pragma unroll
        for (int r = 0; p + r < 3; ++r)
#pragma unroll
          for (int d = 0; d < TK; ++d) ak[d] = mfma16(f[d][0], pf[r], ak[d]);
      }
    }
    same += __shfl_xor(same, 16, 64);
    same += __shfl_xor(same, 32, 64);
    float dot = 0.0f;
#pragma unroll
    for (int d = 0; d < TK; ++d) {
      const floatx4 uv = ru[d].values();
      const floatx4 qv = values4<NP>(lds.x[0] + at<W>(ti, 16 * d + 4 * g), C * W);
      dot += ak[d].x * uv.x + ak[d].y * uv.y + ak[d].z * uv.z + ak[d].w * uv.w;
      ak[d] += same * qv;
    }
    dot += __shfl_xor(dot, 16, 64);
    dot += __shfl_xor(dot, 32, 64);
    if (t < len) {
      if (a.dots && g == 0) a.dots[chain * len + t] = dot;
#pragma unroll
      for (int d = 0; d < TV; ++d) __builtin_nontemporal_store(av[d], reinterpret_cast<floatx4*>(dv + t * DV + 16 * d + 4 * g));
#pragma unroll
      for (int d = 0; d < TK; ++d) __builtin_nontemporal_store(ak[d], reinterpret_cast<floatx4*>(dk + t * DK + 16 * d + 4 * g));
    }
    __builtin_amdgcn_sched_barrier(0);
    st.update(lds);
  }
  if (a.dS0 && step == sp.segs - 1) st.store(a.dS0 + chain * state, DK, 1);
}

// Up to 64 columns: both directions' states, and all three gradients, in one launch each:
// one launch's last workgroups leave no part of the GPU idle.
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
__global__ __launch_bounds__(NT, sizeof(T) == 2 ? 2 : 1) void gradients_kernel(ChunkArgs q, KVArgs kv, Span s, Span r) {
  extern __shared__ __align__(16) unsigned char smem[];
  // the longer work first: the shorter fills what its last workgroups leave idle
  // (8x12x2048x64: 152 us a call against 160 with the two of a segment side by side)
  const long n = q.chains * s.segs, n8 = (n + 7) / 8 * 8;
  const bool second = blockIdx.x >= n8;
  const long unit = second ? blockIdx.x - n8 : blockIdx.x;
  if (unit >= n) return;
  if (!second) kv_body<T, DK, DV>(kv, r, unit, smem);
  else chunk_body<T, float, T, DV, DK, false, true>(q, s, 0, unit, smem);
}
template <typename T, int DK, int DV>
hipError_t both(const ChunkArgs& S, const ChunkArgs& R, const ChunkArgs& q, const KVArgs& kv,
                const Span& s, const Span& r, hipStream_t stream) {
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
  constexpr size_t b1 = sizeof(LdsKV<T, DK, DV>), b2 = sizeof(Lds<T, T, DV, DK>);
  constexpr size_t bytes = b1 > b2 ? b1 : b2;
  auto kernel = gradients_kernel<T, DK, DV>;
  if ((e = lds_limit(kernel, bytes)) != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(grid_of(2, S.chains * s.segs)), dim3(NT), bytes, stream, q, kv, s, r);
  return hipGetLastError();
}
// The same with a size of 128, in blocks of B columns: dk, dq and dv one after the other.
template <typename T, int DK, int DV, int B>
struct Wide {
  static constexpr int BK = DK < B ? DK : B, BV = DV < B ? DV : B, NK = DK / BK, NV = DV / BV;
  static constexpr size_t a = sizeof(Lds<float, T, DV, BK>), b = sizeof(Lds<T, T, DV, BK>),
                          c = sizeof(Lds<T, float, DK, BV>);
  static constexpr size_t bytes = a > b ? (a > c ? a : c) : (b > c ? b : c);
  static constexpr int held = sizeof(T) == 2 && 2 * bytes <= 163840 ? 2 : 1;     // on a compute unit
};
template <typename T, int DK, int DV, int B>
__global__ __launch_bounds__(NT) void wide_states_kernel(ChunkArgs S, Span s, ChunkArgs R, Span r) {
  extern __shared__ __align__(16) unsigned char smem[];
  using X = Wide<T, DK, DV, B>;
  int blk;
  long unit;
  const long ns = S.chains * s.writes, nr = R.chains * r.writes;
  if (!place(2 * X::NV, ns > nr ? ns : nr, blk, unit)) return;
  if (blk < X::NV) {
    if (unit < ns) state_body<T, T, DK, X::BV, false>(S, s, blk, unit, smem);
  } else {
    if (unit < nr) state_body<T, float, DK, X::BV, true>(R, r, blk - X::NV, unit, smem);
  }
}
template <typename T, int DK, int DV, int B>
__global__ __launch_bounds__(NT, (Wide<T, DK, DV, B>::held)) void wide_gradients_kernel(
    ChunkArgs q, ChunkArgs k, ChunkArgs v, Span s, Span r) {
  extern __shared__ __align__(16) unsigned char smem[];
  using X = Wide<T, DK, DV, B>;
  const long n = q.chains * s.segs, n8 = (n + 7) / 8 * 8;
  const int role = (int)(blockIdx.x / n8);
  const long unit = blockIdx.x % n8;
  if (unit >= n) return;
  if (role < X::NK) chunk_body<float, T, T, DV, X::BK, true, true>(k, r, role, unit, smem);
  else if (role < 2 * X::NK) chunk_body<T, float, T, DV, X::BK, false, true>(q, s, role - X::NK, unit, smem);
  else chunk_body<T, T, float, DK, X::BV, true, false>(v, r, role - 2 * X::NK, unit, smem);
}
template <typename T, int DK, int DV, int B>
hipError_t wide(const ChunkArgs& S, const ChunkArgs& R, const ChunkArgs& q, const ChunkArgs& k,
                const ChunkArgs& v, const Span& s, const Span& r, hipStream_t stream) {
  using X = Wide<T, DK, DV, B>;
  hipError_t e;
  const long writes = s.writes > r.writes ? s.writes : r.writes;
  if (writes > 0) {
    constexpr size_t bytes = sizeof(LdsState<T, float, DK, X::BV>);
    auto kernel = wide_states_kernel<T, DK, DV, B>;
    if ((e = lds_limit(kernel, bytes)) != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(grid_of(2 * X::NV, S.chains * writes)), dim3(NT), bytes, stream, S, s, R, r);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if ((e = launch_segments(S.U0, s, R.U0, r, S.chains, (long)DK * DV, stream)) != hipSuccess) return e;
  }
  auto kernel = wide_gradients_kernel<T, DK, DV, B>;
  if ((e = lds_limit(kernel, X::bytes)) != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(grid_of(2 * X::NK + X::NV, S.chains * s.segs)), dim3(NT), X::bytes, stream,
                     q, k, v, s, r);
  return hipGetLastError();
}

// f(dk, dv) as constants: both up to 64, or one of them 128
template <bool WIDE, class F>
hipError_t with_dims(int dk, int dv, F&& f) {
  auto cols = [&](auto k) {
    constexpr bool big = decltype(k)::value == 128;
    switch (dv) {
      case 16: if constexpr (big == WIDE) return f(k, std::integral_constant<int, 16>()); break;
      case 32: if constexpr (big == WIDE) return f(k, std::integral_constant<int, 32>()); break;
      case 64: if constexpr (big == WIDE) return f(k, std::integral_constant<int, 64>()); break;
      case 128: if constexpr (WIDE) return f(k, std::integral_constant<int, 128>()); break;
    }
    return hipErrorInvalidValue;
  };
  switch (dk) {
    case 16: return cols(std::integral_constant<int, 16>());
    case 32: return cols(std::integral_constant<int, 32>());
    case 64: return cols(std::integral_constant<int, 64>());
    case 128: if constexpr (WIDE) return cols(std::integral_constant<int, 128>()); break;
  }
  return hipErrorInvalidValue;
}

// Columns of a block at most with a size of 128.  bf16 with dk >= 64: 32 columns leave room
// for two workgroups on a compute unit, 64 for one (4x16x2048x128: 318 us against 354,
// 8x16x1024x128x64: 164 against 212); with dk 16 and 32 there is room for two of 64
// (8x16x1024x16x128: 110 against 130 us of 32), with float32 inputs for one of either
// (2x16x2048x128: 310 against 366 us).
template <typename T>
constexpr int most_columns(int dk) { return sizeof(T) == 2 && dk >= 64 ? 32 : 64; }

// The two spans of a call (states first token first, their gradients last token first)
// and its workspace.
struct Plan {
  Span s, r;
  int block;               // columns of a workgroup at most; 0: all
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
  // up to 64 columns dk and dv are one workgroup's
  const bool is_wide = a.ndk > 64 || a.ndv > 64;
  const int most = a.dtype == 0 ? most_columns<uint16_t>(a.ndk) : most_columns<float>(a.ndk);
  auto block_for = [&](long whole) {
    const int rows = rows_of(128, p.chains, a.seqlen, whole);
    return rows < most ? rows : most;
  };
  long whole = is_wide ? kWholeWide : kWholeFew, walks = 2 * p.chains;
  if (is_wide) {
    const int b = block_for(1l << 40);
    walks = p.chains * (2 * ((a.ndk + b - 1) / b) + (a.ndv + b - 1) / b);
  }
  if (walks >= kMany) whole = walks >= kMost ? kMostChunks + 1 : kWholeMany;
  p.block = is_wide ? block_for(whole) : 0;
  p.blocks = p.block && p.block < a.ndk ? a.ndk / p.block : 1;
  p.s = cut(p.chains * p.blocks, a.seqlen, 512, kMostChunks, whole);
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
  if (p.block == 0) {
    e = with_dims<false>(a.ndk, a.ndv, [&](auto nk, auto nv) {
      const KVArgs kv{a.q, a.k, a.v, a.dO, a.log_a, a.dS_L, a.dk, a.dv, a.dS0, c, p.chains, a.seqlen};
      return both<T, decltype(nk)::value, decltype(nv)::value>(S, R, dq, kv, p.s, p.r, stream);
    });
  } else {
    e = with_dims<true>(a.ndk, a.ndv, [&](auto nk, auto nv) {
      constexpr int DK = decltype(nk)::value, DV = decltype(nv)::value;
      switch (p.block) {
        case 16: return wide<T, DK, DV, 16>(S, R, dq, dk, dv, p.s, p.r, stream);
        case 32: return wide<T, DK, DV, 32>(S, R, dq, dk, dv, p.s, p.r, stream);
        case 64:
          if constexpr (most_columns<T>(DK) == 64) return wide<T, DK, DV, 64>(S, R, dq, dk, dv, p.s, p.r, stream);
      }
      return hipErrorInvalidValue;
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
