// falcon_gated.hip - forward of the gated linear recurrence over a sequence:
//   S_t = a_t S_{t-1} + v_t k_t^T,   o_t = S_t q_t,   a = exp(log_a)
// in chunks of 64 tokens.  With D_ts = prod_{s<r<=t} a_r, e_t = D_{t,-1}, w_s = D_{63,s}:
//   o_t = e_t S q_t + sum_{s<=t} D_ts (k_s . q_t) v_s
//   S  <- e_63 S + sum_s w_s v_s k_s^T
//
// Work.  A workgroup (4 waves) takes one segment of one chain for up to 64 value rows
// and walks its chunks in order; wave w owns tokens 16w..16w+15 of the chunk for the
// readout, and a part of the state (16 value rows at 64) for the update, which stays in
// its accumulators over the whole segment.  All products are 16x16x32 bf16 MFMA over
// planes (falcon_gated.h).  The scores are formed as P^T = K Q^T: a lane then holds 8
// scores of one token q_t, with the k rows taken in such an order that these are the 8
// k-slots the next product (V^T P^T) wants, so decays, mask and split happen in registers.
// A chunk's k (by rows and transposed), v (transposed) and the state's planes lie in LDS;
// the next chunk's rows are loaded while this one is computed.
//
// Long sequences and few chains.  A sequence is cut into segments until some 768
// workgroups run: a first kernel forms each segment's own write to the state from zero
// (k and v only), a second runs the short recurrence over segments, and the main kernel
// starts each segment from its state.
#include "falcon_gated.h"

namespace falcon {
namespace {

using namespace gated;

template <typename T, int DK, int DVB>
struct Lds {
  static constexpr int NP = planes<T>();
  static constexpr int WK = DK < 32 ? 32 : DK;      // k-slots come in 32s: zeros behind 16
  uint16_t kn[NP][C * WK];                          // k by rows
  uint16_t kt[NP][DK * C];                          // k by columns
  uint16_t vt[NP][DVB * C];                         // v by columns
  uint16_t s[3][DVB * WK];                          // the state at the chunk's start
  double g[C];                                      // G_t
  float e[C], w[C];                                 // 2^G_t, 2^(G_63 - G_t)
};
// what the segments' own writes need
template <typename T, int DK, int DVB>
struct LdsState {
  static constexpr int NP = planes<T>();
  uint16_t kt[NP][DK * C];
  uint16_t vt[NP][DVB * C];
  double g[C];
  float e[C], w[C];
};

// The workgroup's state: wave w holds value rows 16 (w % NDT).. and NK key tiles of 16.
// A lane's part of a tile: value row lane % 16, key columns 4 (lane / 16) + 0..3.
template <int DK, int DVB>
struct State {
  static constexpr int NDT = DVB / 16, WPD = 4 / NDT, ND = DK / 16, NK = (ND + WPD - 1) / WPD;
  floatx4 t[NK];
  static __device__ __forceinline__ int row() { return 16 * ((threadIdx.x >> 6) % NDT) + (threadIdx.x & 15); }
  static __device__ __forceinline__ int tile(int j) { return ((threadIdx.x >> 6) / NDT) * NK + j; }
  static __device__ __forceinline__ int col(int j) { return 16 * tile(j) + 4 * ((threadIdx.x & 63) >> 4); }
  static __device__ __forceinline__ bool has(int j) { return ND % NK == 0 && WPD * NK == ND ? true : tile(j) < ND; }

  __device__ __forceinline__ void load(const float* S) {      // S: row 0 of the block, or null
#pragma unroll
    for (int j = 0; j < NK; ++j)
      t[j] = S && has(j) ? *reinterpret_cast<const floatx4*>(S + row() * DK + col(j))
                         : floatx4{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void store(float* S) const {
#pragma unroll
    for (int j = 0; j < NK; ++j)
      if (has(j)) *reinterpret_cast<floatx4*>(S + row() * DK + col(j)) = t[j];
  }
  template <int W>
  __device__ __forceinline__ void to_planes(uint16_t (*s)[DVB * W]) const {
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      if (!has(j)) continue;
      uint2 h, m, l;
      split3(t[j].x, t[j].y, h.x, m.x, l.x);
      split3(t[j].z, t[j].w, h.y, m.y, l.y);
      const int i = at<W>(row(), col(j));
      *reinterpret_cast<uint2*>(s[0] + i) = h;
      *reinterpret_cast<uint2*>(s[1] + i) = m;
      *reinterpret_cast<uint2*>(s[2] + i) = l;
    }
  }
  // t <- e_63 t + sum_s w_s v_s k_s^T
  template <class L>
  __device__ __forceinline__ void update(const L& lds) {
    constexpr int NP = L::NP;
    const int lane = threadIdx.x & 63, m = lane & 15, g8 = 8 * (lane >> 4);
    const float dec = lds.e[C - 1];
#pragma unroll
    for (int j = 0; j < NK; ++j) t[j] *= dec;
#pragma unroll
    for (int kk = 0; kk < C; kk += 32) {
      bf16x8 v[NP], vw[3];
      float x[8], w[8];
      frag<NP, C>(lds.vt[0], DVB * C, row(), kk + g8, v);
      values<NP>(v, x);
      *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(lds.w + kk + g8);
      *reinterpret_cast<float4*>(w + 4) = *reinterpret_cast<const float4*>(lds.w + kk + g8 + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= w[e];
      frag3(x, vw);
      bf16x8 k[NK][NP];
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        const int tj = has(j) ? tile(j) : 0;
        frag<NP, C>(lds.kt[0], DK * C, 16 * tj + m, kk + g8, k[j]);
      }
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int q = 0; p + q < 3; ++q)
#pragma unroll
          for (int j = 0; j < NK; ++j) t[j] = mfma16(k[j][p], vw[q], t[j]);
    }
  }
};

// Wave 0's sums of the log decays of a chunk, and their place in LDS.
struct Decays {
  double G;
  __device__ __forceinline__ void sum(double x) { G = wave_scan(x); }
  template <class L>
  __device__ __forceinline__ void store(L& lds) const {
    const int lane = threadIdx.x & 63;
    lds.g[lane] = G;
    lds.e[lane] = exp2_of(G);
    lds.w[lane] = exp2_of(__shfl(G, 63, 64) - G);
  }
};

// What one launch works on.
struct Span {
  int chunks;            // of a segment
  int segs;              // segments of a chain
  float* states;         // [chain][segs][dv dk]: segment j's own write in slot j + 1, then
                         // every segment's start (slot 0: S0, so that the last segment
                         // may write S_out over S0)
  float* decays;         // [chain][segs - 1]: segment j's decay
};

template <typename T, int DK, int DVB>
__global__ __launch_bounds__(NT) void gated_state_kernel(GatedArgs a, Span sp) {
  extern __shared__ __align__(16) unsigned char smem[];
  using L = LdsState<T, DK, DVB>;
  L& lds = *reinterpret_cast<L*>(smem);
  int blk;
  long unit;
  if (!place(a.dv / DVB, (long)a.batch * a.heads * (sp.segs - 1), blk, unit)) return;
  const long chain = unit / (sp.segs - 1);
  const int seg = (int)(unit % (sp.segs - 1));
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const long len = a.seqlen, t0 = (long)seg * sp.chunks * C;     // whole chunks all
  const T* k = static_cast<const T*>(a.k) + chain * len * DK;
  const T* v = static_cast<const T*>(a.v) + chain * len * a.dv + blk * DVB;
  const float* la = a.log_a ? a.log_a + chain * len : nullptr;

  Stage<T, DK> sk;
  Stage<T, DVB> sv;
  State<DK, DVB> st;
  Decays dec;
  double total = 0.0;
  st.load(nullptr);
  sk.load(k, t0, len, DK);
  sv.load(v, t0, len, a.dv);
  dec.sum(wave == 0 ? log2_decay(la, t0 + lane, len) : 0.0);
  for (int c = 0; c < sp.chunks; ++c) {
    if (c) __syncthreads();
    sk.template store<C>(nullptr, lds.kt[0]);
    sv.template store<C>(nullptr, lds.vt[0]);
    if (wave == 0) {
      dec.store(lds);
      total += __shfl(dec.G, 63, 64);
    }
    __syncthreads();
    if (c + 1 < sp.chunks) {
      const long t = t0 + (long)(c + 1) * C;
      sk.load(k, t, len, DK);
      sv.load(v, t, len, a.dv);
      if (wave == 0) dec.sum(log2_decay(la, t + lane, len));
    }
    st.update(lds);
  }
  st.store(sp.states + ((chain * sp.segs + seg + 1) * a.dv + (long)blk * DVB) * DK);
  if (threadIdx.x == 0 && blk == 0) sp.decays[unit] = exp2_of(total);
}

// The recurrence over segments: start of segment j + 1 = decay_j start_j + write_j,
// n = segments - 1.  (A call is only cut with fewer than 768 chains.)
__global__ __launch_bounds__(256) void gated_segments_kernel(const float* S0, float* states,
                                                             const float* decays, int n, long size4) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  const long chain = blockIdx.y;
  if (i >= size4) return;
  float4* s = reinterpret_cast<float4*>(states) + chain * (n + 1) * size4 + i;
  const float* d = decays + chain * n;
  float4 x = {0.f, 0.f, 0.f, 0.f};
  if (S0) x = reinterpret_cast<const float4*>(S0)[chain * size4 + i];
  *s = x;
  s += size4;
  for (int j0 = 0; j0 < n; j0 += 8) {
    float4 w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j0 + j < n) w[j] = s[(j0 + j) * size4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j0 + j < n) {
        const float a = d[j0 + j];
        x = float4{a * x.x + w[j].x, a * x.y + w[j].y, a * x.z + w[j].z, a * x.w + w[j].w};
        s[(j0 + j) * size4] = x;
      }
    }
  }
}

template <typename T, int DK, int DVB>
__global__ __launch_bounds__(NT) void gated_fwd_kernel(GatedArgs a, Span sp) {
  extern __shared__ __align__(16) unsigned char smem[];
  using L = Lds<T, DK, DVB>;
  constexpr int NP = L::NP, WK = L::WK, NQ = WK / 32, NDT = DVB / 16;
  L& lds = *reinterpret_cast<L*>(smem);
  int blk;
  long unit;
  if (!place(a.dv / DVB, (long)a.batch * a.heads * sp.segs, blk, unit)) return;
  const long chain = unit / sp.segs;
  const int seg = (int)(unit % sp.segs);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m = lane & 15, g = lane >> 4;
  const long len = a.seqlen, t0 = (long)seg * sp.chunks * C;
  const int chunks = (int)((len - t0 + C - 1) / C) < sp.chunks ? (int)((len - t0 + C - 1) / C) : sp.chunks;
  const T* q = static_cast<const T*>(a.q) + chain * len * DK;
  const T* k = static_cast<const T*>(a.k) + chain * len * DK;
  const T* v = static_cast<const T*>(a.v) + chain * len * a.dv + blk * DVB;
  const float* la = a.log_a ? a.log_a + chain * len : nullptr;
  float* o = a.o + chain * len * a.dv + blk * DVB;
  const long S_at = (chain * a.dv + (long)blk * DVB) * DK;

  Stage<T, DK> sk;
  Stage<T, DVB> sv;
  State<DK, DVB> st;
  Decays dec;
  Raw<T> rq[NQ];
  auto load_q = [&](long base) {
    const long t = base + 16 * wave + m;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      if (t < len && 32 * i + 8 * g < DK) rq[i].load(q + t * DK + 32 * i + 8 * g);
      else rq[i].zero();
    }
  };
  sk.load(k, t0, len, DK);
  sv.load(v, t0, len, a.dv);
  load_q(t0);
  dec.sum(wave == 0 ? log2_decay(la, t0 + lane, len) : 0.0);
  if (sp.segs > 1) st.load(sp.states + (unit * a.dv + (long)blk * DVB) * DK);
  else st.load(a.S0 ? a.S0 + S_at : nullptr);
  if (DK < WK) {      // k-slots behind the last column
    for (int i = threadIdx.x; i < NP * C * WK / 8; i += NT) reinterpret_cast<uint4*>(lds.kn[0])[i] = uint4{0u, 0u, 0u, 0u};
    for (int i = threadIdx.x; i < 3 * DVB * WK / 8; i += NT) reinterpret_cast<uint4*>(lds.s[0])[i] = uint4{0u, 0u, 0u, 0u};
    __syncthreads();
  }

  for (int c = 0; c < chunks; ++c) {
    const long t = t0 + (long)c * C;
    if (c) __syncthreads();
    sk.template store<WK>(lds.kn[0], lds.kt[0]);
    sv.template store<C>(nullptr, lds.vt[0]);
    st.template to_planes<WK>(lds.s);
    if (wave == 0) dec.store(lds);
    bf16x8 qf[NQ][NP];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      uint4 f[NP];
      rq[i].split(f);
#pragma unroll
      for (int p = 0; p < NP; ++p) qf[i][p] = __builtin_bit_cast(bf16x8, f[p]);
    }
    __syncthreads();
    if (c + 1 < chunks) {
      sk.load(k, t + C, len, DK);
      sv.load(v, t + C, len, a.dv);
      load_q(t + C);
      if (wave == 0) dec.sum(log2_decay(la, t + C + lane, len));
    }

    // o^T: value rows x this wave's 16 tokens; first the state's part
    floatx4 acc[NDT];
#pragma unroll
    for (int i = 0; i < NDT; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      bf16x8 s[NDT][3];
#pragma unroll
      for (int d = 0; d < NDT; ++d) frag<3, WK>(lds.s[0], DVB * WK, 16 * d + m, 32 * i + 8 * g, s[d]);
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int r = 0; r < NP; ++r)
          if (p + r < 3) {
#pragma unroll
            for (int d = 0; d < NDT; ++d) acc[d] = mfma16(s[d][p], qf[i][r], acc[d]);
          }
    }
    const int ti = 16 * wave + m;               // this lane's token in the chunk
    const float e = lds.e[ti];
    const double Gt = lds.g[ti];
#pragma unroll
    for (int d = 0; d < NDT; ++d) acc[d] *= e;
    // then the chunk's own tokens, 32 at a time; none behind the wave's last token
#pragma unroll
    for (int kk = 0; kk < C; kk += 32) {
      if (kk > 16 * wave + 15) break;
      float x[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // row m of this tile: token kk + 8 (m / 4) + 4 j + m % 4
        floatx4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          bf16x8 kf[NP];
          frag<NP, WK>(lds.kn[0], C * WK, kk + 8 * (m >> 2) + 4 * j + (m & 3), 32 * i + 8 * g, kf);
          mma<NP, NP>(kf, qf[i], p);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int s = kk + 8 * g + 4 * j + r;
          const float dcy = exp2_of(Gt - lds.g[s]);
          x[4 * j + r] = s <= ti ? p[r] * dcy : 0.0f;
        }
      }
      bf16x8 pf[3];
      frag3(x, pf);
      bf16x8 vf[NDT][NP];
#pragma unroll
      for (int d = 0; d < NDT; ++d) frag<NP, C>(lds.vt[0], DVB * C, 16 * d + m, kk + 8 * g, vf[d]);
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int r = 0; p + r < 3; ++r)
#pragma unroll
          for (int d = 0; d < NDT; ++d) acc[d] = mfma16(vf[d][p], pf[r], acc[d]);
    }
    if (t + ti < len) {
#pragma unroll
      for (int d = 0; d < NDT; ++d)
        *reinterpret_cast<floatx4*>(o + (t + ti) * a.dv + 16 * d + 4 * g) = acc[d];
    }
    st.update(lds);
  }
  if (a.S_out && seg == sp.segs - 1) st.store(a.S_out + S_at);
}

// Value rows of a workgroup: 64, or 32 where the planes of float32 inputs at dk = 128
// would not fit the LDS.
template <typename T, int DK>
constexpr int most_rows() { return sizeof(T) == 4 && DK == 128 ? 32 : 64; }
int rows_of(int dtype, int dk, int dv) {
  const int most = dtype == 1 && dk == 128 ? 32 : 64;
  return dv < most ? dv : most;
}

Segments cut(const GatedArgs& a, bool workspace) {
  const long units = (long)a.batch * a.heads * (a.dv / rows_of(a.dtype, a.dk, a.dv));
  return segments(workspace ? units : 1l << 40, a.seqlen);
}
size_t state_floats(const GatedArgs& a, int segs) {
  return (size_t)a.batch * a.heads * segs * a.dv * a.dk;
}

// A kernel with more than 64 KB of LDS has to be told so, once a device; the call costs
// a microsecond and keeps no state here.
template <class K>
hipError_t lds_limit(K kernel, size_t bytes) {
  if (bytes <= 65536) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int DK, int DVB>
hipError_t go(const GatedArgs& a, const Span& sp, hipStream_t stream) {
  const int blocks = a.dv / DVB;
  const long chains = (long)a.batch * a.heads;
  hipError_t e;
  if (sp.segs > 1) {
    constexpr size_t bytes = sizeof(LdsState<T, DK, DVB>);
    if ((e = lds_limit(gated_state_kernel<T, DK, DVB>, bytes)) != hipSuccess) return e;
    hipLaunchKernelGGL((gated_state_kernel<T, DK, DVB>), dim3(grid_of(blocks, chains * (sp.segs - 1))),
                       dim3(NT), bytes, stream, a, sp);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const long size4 = (long)a.dv * a.dk / 4;
    hipLaunchKernelGGL(gated_segments_kernel, dim3((unsigned)((size4 + 255) / 256), (unsigned)chains),
                       dim3(256), 0, stream, a.S0, sp.states, sp.decays, sp.segs - 1, size4);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  constexpr size_t bytes = sizeof(Lds<T, DK, DVB>);
  if ((e = lds_limit(gated_fwd_kernel<T, DK, DVB>, bytes)) != hipSuccess) return e;
  hipLaunchKernelGGL((gated_fwd_kernel<T, DK, DVB>), dim3(grid_of(blocks, chains * sp.segs)), dim3(NT),
                     bytes, stream, a, sp);
  return hipGetLastError();
}

template <typename T, int DK>
hipError_t with_dv(const GatedArgs& a, const Span& sp, hipStream_t stream) {
  switch (rows_of(a.dtype, a.dk, a.dv)) {
    case 16: return go<T, DK, 16>(a, sp, stream);
    case 32: return go<T, DK, 32>(a, sp, stream);
    case 64:
      if constexpr (most_rows<T, DK>() == 64) return go<T, DK, 64>(a, sp, stream);
  }
  return hipErrorInvalidValue;
}
template <typename T>
hipError_t with_dk(const GatedArgs& a, const Span& sp, hipStream_t stream) {
  switch (a.dk) {
    case 16: return with_dv<T, 16>(a, sp, stream);
    case 32: return with_dv<T, 32>(a, sp, stream);
    case 64: return with_dv<T, 64>(a, sp, stream);
    case 128: return with_dv<T, 128>(a, sp, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

size_t gated_workspace_bytes(const GatedArgs& a) {
  const Segments s = cut(a, true);
  if (s.count == 1) return 0;
  return (state_floats(a, s.count) + (size_t)a.batch * a.heads * (s.count - 1)) * sizeof(float);
}

hipError_t launch_gated(const GatedArgs& a, void* ws, size_t ws_bytes, hipStream_t stream) {
  (void)hipGetLastError();
  const bool use = ws && ws_bytes >= gated_workspace_bytes(a);
  const Segments s = cut(a, use);
  float* states = use ? static_cast<float*>(ws) : nullptr;
  const Span sp{s.chunks, s.count, states, states ? states + state_floats(a, s.count) : nullptr};
  return a.dtype == 0 ? with_dk<uint16_t>(a, sp, stream) : with_dk<float>(a, sp, stream);
}

}  // namespace falcon
