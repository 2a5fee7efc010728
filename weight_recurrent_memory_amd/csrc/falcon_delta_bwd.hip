// falcon_delta_bwd.hip - gradients of the gated delta rule over a sequence.
//
// With R_t the gradient of S_t, o_t's own read in it, and R the one behind a chunk of 64
// tokens (T, D, e, w, d as in falcon_delta.h, P_ts = D_ts q_t . k_s for s <= t):
//   du = T^T (P^T dO + w (K R^T))              gradient of u, last chunk first
//   R <- d R + dO^T (e Q) - (b du)^T (e K)
//   dv = b du
//   dq_t = S_t^T dO_t   = e_t S^T dO_t + sum_{s<=t} D_ts (u_s . dO_t) k_s
//   y_t  = a_t S_{t-1}^T du_t = e_t S^T du_t + sum_{s<t} D_ts (u_s . du_t) k_s
//   dk_t = R_t^T u_t - b_t y_t,  R_t^T u_t = w_t R^T u_t + sum_{s>=t} D_st (dO_s . u_t) q_s
//                                             - sum_{s>t} D_st b_s (du_s . u_t) k_s
//   dbeta_t = du_t . v_t - y_t . k_t
//   dlog_a_t = <a_t (R_t - dv_t k_t^T), S_{t-1}>, what passes the border before t;
//   dlog_a_t - dlog_a_{t+1} = q_t . dq_t - v_t . dv_t, summed in float64 from <R, S'> behind
//   the chunk, S' = d S + sum_s w_s u_s k_s^T.  At a reset it is 0 and the sum begins anew.
//
// Four launches: every chunk's T and its transpose; P^T dO and dO^T (e Q) of every chunk;
// the walks, S and u from the first chunk on and R and du from the last one, side by side,
// both by falcon_delta_walk.h's wave of 16 value rows; every chunk's outputs from S, R, u, du.
//
// 8x12x2048x64 bf16: 32 + 40 + 127 to 132 + 133 to 140 us of kernels, 305 us a call.  The walks
// write S, R, u and du (197 MB) and wait for each other's chunks; without these writes they would take
// 84 us, and the outputs would have no states to start from.  The outputs read and write 460 MB
// (3.5 TB/s) and issue 2030 vector instructions a chunk and wave, 336 of them matrix ones, two
// workgroups a compute unit.  Sequences of few chains in segments, as the forward's: 1x5x4099, 128x64
// 12 + 11 + 24 + 19 + 26 + 40 us, 127 us a call (walked whole 266).  Tried: stores past the caches (128 -> 136 us).
#include "falcon_delta_walk.h"

namespace falcon {
namespace delta {
namespace {

struct BwdArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* beta;
  const float* log_a;      // or null
  const float* S0;         // or null
  const float* dO;
  const float* dS_L;       // or null
  float* dq;
  float* dk;
  float* dv;               // du until the last launch
  float* dbeta;
  float* dlog_a;           // or null
  float* dS0;              // or null
  const uint4* T;
  const uint4* Tt;
  float4* H;               // P^T dO: [chain][chunk][value tile][4][64], a walker's tiles
  float4* G;               // dO^T (e Q): [chain][chunk][value tile][dk / 16][64]
  float* U;                // [chain][L][dv]
  float* S;                // [chain][chunks][dv][dk]: before each chunk
  float* R;                // [chain][chunks][dv][dk]: behind each chunk
  long chains;
  int seqlen, nv;
  // segments of a chain, chunks of one; with several, what each walk starts from (Joins of the
  // two directions; a segment is a step, the last one the backward walk's first)
  int segs, per;
  float* starts_S;
  float* starts_R;
  uint4* moves;            // [chain][segs][StateT::kMove]: what a segment multiplies its start's rows with
  uint4* moves_t;          // the same for R
};

// ----------------------------------------------- P^T dO and dO^T (e Q)

template <typename T, int DK>
struct PrepLds {
  alignas(16) uint4 p[kFrags][3][64];        // P^T: rows s, slots t
  alignas(16) uint16_t q[planes<T>()][C * DK];
  Gates gate;
};

// One chunk: wave w forms P^T's rows 16 w.., then takes the value tiles w, w + 4.
template <typename T, int DK>
__global__ __launch_bounds__(256) void prep_kernel(BwdArgs a, int chunks) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int NP = planes<T>(), NQ = (DK + 31) / 32, NK = DK / 16;
  PrepLds<T, DK>& lds = *reinterpret_cast<PrepLds<T, DK>*>(smem);
  const int wave = wave_id(), lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const long unit = blockIdx.x, chain = unit / chunks, t0 = (unit % chunks) * C, len = a.seqlen, left = len - t0;
  const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
  const T* q = static_cast<const T*>(a.q) + (chain * len + t0) * DK;
  const T* k = static_cast<const T*>(a.k) + (chain * len + t0) * DK;
  const Window wq(q, left, DK, 0), wk(k, left, DK, 0);
  StageK<T, DK, 256> sq;
  sq.load(wq, threadIdx.x);
  GateLoad gl;
  if (wave == 0) gl.load(a.log_a ? a.log_a + chain * len : nullptr, a.beta + chain * len, t0, len);
  bf16x8 kf[NQ][NP];
  {
    PairRow<T, DK> row;
    row.load(wk, 16 * wave + m);
#pragma unroll
    for (int i = 0; i < NQ; ++i) row.frag(i, kf[i]);
  }
  sq.store(lds.q[0], threadIdx.x);
  if (wave == 0) gl.store(lds.gate);
  __syncthreads();
  const float2 Gs = lds.gate.g[16 * wave + m];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (2 * h + 1 < wave) continue;
    floatx4 p[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int ti = 2 * h + z;
      p[z] = zero;
      if (ti < wave) continue;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        bf16x8 qf[NP];
        pair_frag<NP, DK>(lds.q[0], 16 * ti + m, i, qf);
        mma<NP, NP>(qf, kf[i], p[z]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = p[z][r] * decay(lds.gate.g[16 * ti + 4 * g + r], Gs);
        p[z][r] = (ti > wave || 4 * g + r >= m) ? x : 0.0f;
      }
    }
    bf16x8 f[3];
    frag_pair(p[0], p[1], f);
#pragma unroll
    for (int n = 0; n < 3; ++n) lds.p[frag_of(3 - wave, 1 - h)][n][lane] = __builtin_bit_cast(uint4, f[n]);
  }
  __syncthreads();
  const int tiles = a.nv / 16;
  const float* dO = a.dO + (chain * len + t0) * a.nv;
  const Window wo(dO, left, a.nv, 0);
  for (int z = wave; z < tiles; z += 4) {
    floatx4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[i][r] = load_f32(wo, ((16 * i + 4 * g + r) * a.nv + 16 * z + m) * 4);
    bf16x8 of[2][3];
    frag_pair(o[0], o[1], of[0]);
    frag_pair(o[2], o[3], of[1]);
    float4* H = a.H + (unit * tiles + z) * 4 * 64 + lane;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      floatx4 x = zero;
#pragma unroll
      for (int j = s / 2; j < 2; ++j) {
        bf16x8 f[3];
#pragma unroll
        for (int n = 0; n < 3; ++n) f[n] = __builtin_bit_cast(bf16x8, lds.p[frag_of(3 - s, 1 - j)][n][lane]);
        mma<3, 3>(f, of[j], x);
      }
      *reinterpret_cast<floatx4*>(H + s * 64) = x;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= four(lds.gate.e + 16 * i + 4 * g);
    frag_pair(o[0], o[1], of[0]);
    frag_pair(o[2], o[3], of[1]);
    float4* G = a.G + (unit * tiles + z) * NK * 64 + lane;
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      floatx4 x = zero;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        bf16x8 f[NP];
        pair_frag_t<NP, DK>(lds.q[0], n, j, f);
        mma<NP, 3>(f, of[n], x);
      }
      *reinterpret_cast<floatx4*>(G + j * 64) = x;
    }
  }
}

// ------------------------------------------------------------ the walks

// The wave that walks 16 value rows backward: R in StateT.
template <typename T, int DK>
struct BackWalker {
  static constexpr int NP = planes<T>(), NQ = (DK + 31) / 32, NK = DK / 16;
  StateT<DK> R;
  LdsT t;
  floatx4 h[4], G[NK];

  __device__ __forceinline__ void load_h(const float4* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const floatx4*>(p + i * 64 + (threadIdx.x & 63));
  }
  __device__ __forceinline__ void load_G(const float4* p) {
#pragma unroll
    for (int i = 0; i < NK; ++i) G[i] = *reinterpret_cast<const floatx4*>(p + i * 64 + (threadIdx.x & 63));
  }

  template <class Load, class Load2, class Values>
  __device__ __forceinline__ void chunk(const uint16_t* k, const Gates& gt, Load&& load, Load2&& load2,
                                        Values&& values) {
    const int g = (threadIdx.x & 63) >> 4, m = threadIdx.x & 15;
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    floatx4 x[4] = {zero, zero, zero, zero};
    // K R^T
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      bf16x8 s[3], kn[4][NP];
      R.frag(n, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) pair_frag<NP, DK>(k, 16 * i + m, n, kn[i]);
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int r = 0; p + r < 3; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = mfma16(kn[i][p], s[r], x[i]);
    }
    // Y = H + w K R^T, du = T^T Y
    bf16x8 f[3];
    floatx4 u[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 2 * j; i < 2 * j + 2; ++i) {
        const floatx4 w = four(gt.w + 16 * i + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[i][r] = h[i][r] + w[r] * x[i][r];
      }
      frag_pair(x[2 * j], x[2 * j + 1], f);
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int i = 0; i < 2 * j + 2; ++i) {
          const bf16x8 tf = t.get(frag_of(3 - i, 1 - j), p);
#pragma unroll
          for (int r = 0; p + r < 3; ++r) u[i] = mfma16(tf, f[r], u[i]);
        }
    }
    // (keeps the next part's reads in that part: registers)
    __builtin_amdgcn_sched_barrier(0);
    load();
    values(u);
    // R <- d R + G - (b e du)^T K
    const float d = gt.d;
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) R.t[j][r] = d * R.t[j][r] + G[j][r];
    load2();
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const floatx4 b0 = four(gt.be + 32 * n + 4 * g);
      const floatx4 b1 = four(gt.be + 32 * n + 16 + 4 * g);
      frag_pair(-b0 * u[2 * n], -b1 * u[2 * n + 1], f);
      constexpr int J = NK < 4 ? NK : 4;
#pragma unroll
      for (int j0 = 0; j0 < NK; j0 += J) {
        bf16x8 kt[J][NP];
#pragma unroll
        for (int j = 0; j < J; ++j) pair_frag_t<NP, DK>(k, n, j0 + j, kt[j]);
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int r = 0; p + r < 3; ++r)
#pragma unroll
            for (int j = 0; j < J; ++j) R.t[j0 + j] = mfma16(kt[j][p], f[r], R.t[j0 + j]);
      }
    }
  }
};

// u or du of a chunk's tokens (p: the first one's row), 16 value columns from `col` on; rows
// behind the last token are outside of the window.
__device__ __forceinline__ void store_values(const float* p, int nv, int col, long left, const floatx4 (&u)[4]) {
  const int g = (threadIdx.x & 63) >> 4, m = threadIdx.x & 15;
  const Window w(p, left, nv, 0);
  const int first = (4 * g * nv + col + m) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float x = u[i][r];         // (a bit cast of a vector's element takes the first one's bits)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), w.r, first + (16 * i + r) * nv * 4, 0, 0);
    }
}

// ND walkers of one segment; the first blocks walk forward, as many more backward.  WRITE: each
// segment's own write from zero, and forward, behind the value rows, unit rows, which give the matrix
// that a segment multiplies its start's rows with.
template <typename T, int DK, int ND, bool WRITE>
__global__ __launch_bounds__(64 * (ND + kKeyWaves), 2) void walks_kernel(BwdArgs a, int chunks) {
  extern __shared__ __align__(16) unsigned char smem[];
  using L = KeyLds<T, DK>;
  constexpr int DZ = 16 * ND, NK = DK / 16;
  L& lds = *reinterpret_cast<L*>(smem);
  const int ahead = WRITE ? write_blocks(a.nv + DK) : a.nv / DZ;
  int blk;
  long unit;
  if (!place(ahead + (WRITE ? write_blocks(a.nv) : a.nv / DZ), a.chains * a.segs, blk, unit)) return;
  const long chain = unit / a.segs;
  const int seg = (int)(unit % a.segs);
  const bool back = blk >= ahead;
  const int wave = wave_id();
  const long c0 = (long)seg * a.per, first = chain * a.seqlen + c0 * C, left = a.seqlen - c0 * C;
  const int n = chunks - c0 < a.per ? (int)(chunks - c0) : a.per;
  if (wave >= ND) {
    const T* k = static_cast<const T*>(a.k) + first * DK;
    const float* la = a.log_a ? a.log_a + first : nullptr;
    if (back) keys_only<T, DK, true>(lds, k, la, a.beta + first, a.Tt + (chain * chunks + c0) * kT, left, n, threadIdx.x - 64 * ND);
    else keys_only<T, DK, false>(lds, k, la, a.beta + first, a.T + (chain * chunks + c0) * kT, left, n, threadIdx.x - 64 * ND);
    return;
  }
  const int from = (back ? blk - ahead : blk) * DZ + 16 * wave;
  const bool unit_rows = WRITE && !back && from >= a.nv;
  const int row = unit_rows ? from - a.nv : from;
  if (WRITE && row >= (unit_rows ? DK : a.nv)) return idle(n);
  const long state = (long)a.nv * DK, at = (long)row * DK;
  if (!back) {
    Walker<T, DK, LdsT> w;
    const T* v = static_cast<const T*>(a.v) + first * a.nv;
    float* S = a.S + (chain * chunks + c0) * state + at;
    const float* U = a.U + first * a.nv;
    if (unit_rows) w.S.unit(row);
    else if (WRITE) w.S.load(nullptr);
    else if (a.segs > 1) w.S.load(a.starts_S + unit * state + at);
    else w.S.load(a.S0 ? a.S0 + chain * state + at : nullptr);
    auto load_v = [&](int c) {
      w.load_v(v + (long)c * C * a.nv, unit_rows ? 0 : left - (long)c * C, a.nv, row);
    };
    load_v(0);
    for (int c = 0; c < n; ++c) {
      __syncthreads();
      if (c == 0) w.load_k(lds.k[0][0]);
      const int next = c + 1 < n ? c + 1 : c;
      if (!WRITE) w.S.store(S + c * state);
      w.t.p = lds.t[c & 1];
      w.chunk(lds.k[c % L::R][0], lds.gate[c % L::R],
              [&] { load_v(next); },
              [&] { w.load_k(lds.k[next % L::R][0]); }, [](int, int, const bf16x8&) {},
              [&](const floatx4 (&u)[4]) {
                if (!WRITE) store_values(U + (long)c * C * a.nv, a.nv, row, left - (long)c * C, u);
              },
              [](int, const floatx4 (&)[4]) {});
    }
    __syncthreads();
    if (!WRITE) return;
    if (unit_rows) {
      w.S.store_moves(a.moves + unit * StateT<DK>::kMove, a.moves_t + unit * StateT<DK>::kMove, row / 16);
    } else if (seg < a.segs - 1) {
      w.S.store(a.starts_S + (unit + 1) * state + at);
    }
    return;
  }
  BackWalker<T, DK> w;
  const int tiles = a.nv / 16, z = row / 16;
  const float4* H = a.H + ((chain * chunks + c0) * tiles + z) * 4 * 64;
  const float4* G = a.G + ((chain * chunks + c0) * tiles + z) * NK * 64;
  float* R = a.R + (chain * chunks + c0) * state + at;
  const float* du = a.dv + first * a.nv;
  const long step = chain * a.segs + a.segs - 1 - seg;
  if (WRITE) w.R.load(nullptr);
  else if (a.segs > 1) w.R.load(a.starts_R + step * state + at);
  else w.R.load(a.dS_L ? a.dS_L + chain * state + at : nullptr);
  w.load_h(H + (long)(n - 1) * tiles * 4 * 64);
  w.load_G(G + (long)(n - 1) * tiles * NK * 64);
  for (int i = 0; i < n; ++i) {
    __syncthreads();
    const int c = n - 1 - i, next = c > 0 ? c - 1 : 0;
    if (!WRITE) w.R.store(R + c * state);
    w.t.p = lds.t[i & 1];
    w.chunk(lds.k[i % L::R][0], lds.gate[i % L::R],
            [&] { w.load_h(H + (long)next * tiles * 4 * 64); },
            [&] { w.load_G(G + (long)next * tiles * NK * 64); },
            [&](const floatx4 (&u)[4]) {
              if (!WRITE) store_values(du + (long)c * C * a.nv, a.nv, row, left - (long)c * C, u);
            });
  }
  __syncthreads();
  if (WRITE) {
    if (seg > 0) w.R.store(a.starts_R + (step + 1) * state + at);
  } else if (a.dS0 && seg == 0) {
    w.R.store(a.dS0 + chain * state + at);
  }
}

// --------------------------------------------------------------- outputs

constexpr int kSlice = 32;           // value columns at a time

template <typename T, int DK>
struct OutLds {
  static constexpr int NP = planes<T>();
  struct Slice {
    uint16_t u[3][C * kSlice], o[3][C * kSlice], d[3][C * kSlice];
    uint16_t s[3][kSlice * DK], r[3][kSlice * DK];
  };
  struct Rows {
    uint16_t k[NP][C * DK], q[NP][C * DK];
  };
  union {
    alignas(16) Slice a;             // first
    alignas(16) Rows b;              // behind the last slice
  };
  Gates gate;
  alignas(16) float step[C];
  alignas(16) double x[4];
};

// Offset of a slice's row and 16-byte group in LDS: rows of 64 bytes, so rows 4 apart meet in
// their banks; the groups are XORed by that, and 16 rows' reads of one group fall apart.
__device__ __forceinline__ int slice_at(int row, int group) { return row * kSlice + ((group ^ ((row >> 2) & 3)) << 3); }
__device__ __forceinline__ void slice_frag(const uint16_t* p, int row, bf16x8 (&f)[3]) {
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int n = 0; n < 3; ++n) f[n] = frag_bf16(p + n * C * kSlice + slice_at(row, g));
}

// 64 rows of kSlice columns of a [token][nv] array, 8 of a row a thread.
struct StageValues {
  Raw<float> r;
  __device__ __forceinline__ void load(const Window& w, int nv, int col) {
    const int c = col + 8 * (threadIdx.x & 3);
    r.load(w, c < nv ? ((threadIdx.x >> 2) * nv + c) * 4 : kNowhere);
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
    uint4 f[3];
    r.split(f);
#pragma unroll
    for (int n = 0; n < 3; ++n)
      *reinterpret_cast<uint4*>(p + n * C * kSlice + slice_at(threadIdx.x >> 2, threadIdx.x & 3)) = f[n];
  }
};
// kSlice rows of a state.
template <int DK>
struct StageState {
  static constexpr int G = DK / 8, UNITS = kSlice * G, N = (UNITS + 255) / 256;
  Raw<float> r[N];
  __device__ __forceinline__ void load(const float* S, int rows) {
    const Window w(S, rows < kSlice ? rows : kSlice, DK, 0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = threadIdx.x + 256 * i;
      r[i].load(w, UNITS % 256 == 0 || u < UNITS ? 32 * u : kNowhere);
    }
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = threadIdx.x + 256 * i;
      if (UNITS % 256 != 0 && u >= UNITS) continue;
      uint4 f[3];
      r[i].split(f);
#pragma unroll
      for (int n = 0; n < 3; ++n)
        *reinterpret_cast<uint4*>(p + n * kSlice * DK + at<DK>(u / G, 8 * (u % G))) = f[n];
    }
  }
  __device__ __forceinline__ double dot(const StageState& o) const {
    double x = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const floatx4 a = __builtin_bit_cast(floatx4, r[i].a), b = __builtin_bit_cast(floatx4, r[i].b);
      const floatx4 c = __builtin_bit_cast(floatx4, o.r[i].a), d = __builtin_bit_cast(floatx4, o.r[i].b);
#pragma unroll
      for (int j = 0; j < 4; ++j) x += (double)a[j] * c[j] + (double)b[j] * d[j];
    }
    return x;
  }
};

// Four values of NP planes in LDS.
template <int NP>
__device__ __forceinline__ floatx4 row_values(const uint16_t* p, int stride) {
  floatx4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = NP - 1; i >= 0; --i) {
    Raw4<uint16_t> r;
    r.u = *reinterpret_cast<const uint2*>(p + i * stride);
    x += r.values();
  }
  return x;
}

// One chunk; wave w owns tokens 16 w.. (as columns m of its results).  (Eight waves, half of them
// for the rows behind a token, hold one chunk a compute unit in place of two: 181 us against 143
// at 8x12x2048x64.)
template <typename T, int DK>
__global__ __launch_bounds__(256, (DK <= 64 ? 2 : 1)) void outputs_kernel(BwdArgs a, int chunks) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int NP = planes<T>(), NK = DK / 16;
  OutLds<T, DK>& lds = *reinterpret_cast<OutLds<T, DK>*>(smem);
  const int wave = wave_id(), lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const long unit = blockIdx.x, chain = unit / chunks, len = a.seqlen;
  const int chunk = (int)(unit % chunks);
  const long t0 = (long)chunk * C, left = len - t0, row = chain * len + t0;
  const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
  const long state = (long)a.nv * DK;
  const Window wu(a.U + row * a.nv, left, a.nv, 0), wo(a.dO + row * a.nv, left, a.nv, 0),
      wd(a.dv + row * a.nv, left, a.nv, 0);
  const float* S = a.S + (chain * chunks + chunk) * state;
  const float* R = a.R + (chain * chunks + chunk) * state;
  const T* v = static_cast<const T*>(a.v) + row * a.nv;
  const Window wv(v, left, a.nv, 0);

  StageValues su, so, sd;
  StageState<DK> ss, sr;
  GateLoad gl;
  Raw<T> rv;
  auto fetch = [&](int col) {
    su.load(wu, a.nv, col);
    so.load(wo, a.nv, col);
    sd.load(wd, a.nv, col);
    ss.load(S + (long)col * DK, a.nv - col);
    sr.load(R + (long)col * DK, a.nv - col);
    rv.load(wv, col + 8 * (threadIdx.x & 3) < a.nv
                    ? ((threadIdx.x >> 2) * a.nv + col + 8 * (threadIdx.x & 3)) * (int)sizeof(T) : kNowhere);
  };
  fetch(0);
  if (wave == 0) {
    gl.load(a.log_a ? a.log_a + chain * len : nullptr, a.beta + chain * len, t0, len);
    gl.store(lds.gate);
  }
  // scores by tiles j: j < w: rows s of u, columns t of dO and du; j > w: rows t of dO and
  // du, columns of u; j == w: both
  floatx4 Z[4], W[4], Zd = zero, Wd = zero, dq[NK], y[NK], dk[NK];
#pragma unroll
  for (int j = 0; j < 4; ++j) Z[j] = W[j] = zero;
#pragma unroll
  for (int j = 0; j < NK; ++j) dq[j] = y[j] = dk[j] = zero;
  StageK<T, DK, 256> sk, sq;
  const Window wk(static_cast<const T*>(a.k) + row * DK, left, DK, 0),
      wq(static_cast<const T*>(a.q) + row * DK, left, DK, 0);
  float duv = 0.0f;                  // of token threadIdx.x / 4: du . v over this thread's columns
  double X = 0.0;                    // <R, S> of this thread's part
  for (int col = 0; col < a.nv; col += kSlice) {
    if (col) __syncthreads();
    su.store(lds.a.u[0]);
    so.store(lds.a.o[0]);
    sd.store(lds.a.d[0]);
    ss.store(lds.a.s[0]);
    sr.store(lds.a.r[0]);
    if (a.dlog_a) X += sr.dot(ss);
    __syncthreads();
    // dv = b du, and du . v
    {
      const float b = lds.gate.b[threadIdx.x >> 2];
      const floatx4 lo = __builtin_bit_cast(floatx4, sd.r.a), hi = __builtin_bit_cast(floatx4, sd.r.b);
      float x[8];
      uint4 f[planes<T>()];
      rv.split(f);
      bf16x8 fb[planes<T>()];
#pragma unroll
      for (int n = 0; n < planes<T>(); ++n) fb[n] = __builtin_bit_cast(bf16x8, f[n]);
      values<planes<T>()>(fb, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) duv += lo[j] * x[j] + hi[j] * x[4 + j];
      const int t = threadIdx.x >> 2, c = col + 8 * (threadIdx.x & 3);
      if (t < left && c < a.nv) {
        float* p = a.dv + (row + t) * a.nv + c;
        *reinterpret_cast<floatx4*>(p) = b * lo;
        *reinterpret_cast<floatx4*>(p + 4) = b * hi;
      }
    }
    if (col + kSlice < a.nv) {
      fetch(col + kSlice);
    } else if (planes<T>() == 1) {
      sk.load(wk, threadIdx.x);
      sq.load(wq, threadIdx.x);
    }
    bf16x8 uf[3], of[3], df[3];
    slice_frag(lds.a.u[0], 16 * wave + m, uf);
    slice_frag(lds.a.o[0], 16 * wave + m, of);
    slice_frag(lds.a.d[0], 16 * wave + m, df);
    mma<3, 3>(uf, of, Zd);
    mma<3, 3>(uf, df, Wd);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x8 f[3];
      if (j < wave) {
        slice_frag(lds.a.u[0], 16 * j + m, f);
        mma<3, 3>(f, of, Z[j]);
        mma<3, 3>(f, df, W[j]);
      } else {
        slice_frag(lds.a.o[0], 16 * j + m, f);
        mma<3, 3>(f, uf, Z[j]);
        slice_frag(lds.a.d[0], 16 * j + m, f);
        mma<3, 3>(f, uf, W[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      bf16x8 f[3];
      frag_t<3, DK>(lds.a.s[0], kSlice * DK, 8 * g, 16 * j, f);
      mma<3, 3>(f, of, dq[j]);
      mma<3, 3>(f, df, y[j]);
      frag_t<3, DK>(lds.a.r[0], kSlice * DK, 8 * g, 16 * j, f);
      mma<3, 3>(f, uf, dk[j]);
    }
  }
  // K and Q in the slices' place
  if (planes<T>() > 1) {
    sk.load(wk, threadIdx.x);
    sq.load(wq, threadIdx.x);
  }
  __syncthreads();
  sk.store(lds.b.k[0], threadIdx.x);
  sq.store(lds.b.q[0], threadIdx.x);
  duv += __shfl_xor(duv, 1, 64);
  duv += __shfl_xor(duv, 2, 64);
  if ((threadIdx.x & 3) == 0) lds.step[threadIdx.x >> 2] = duv;
  __syncthreads();

  const int ti = 16 * wave + m;      // this lane's token
  if (a.dlog_a) {
    // what passes the border behind the chunk: <R, d S + sum_s w_s u_s k_s^T>, of which
    // k_s . (R^T u_s) is on the way to dk
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const floatx4 kv = row_values<NP>(lds.b.k[0] + at<DK>(ti, 16 * j + 4 * g), C * DK);
#pragma unroll
      for (int r = 0; r < 4; ++r) sum += (double)kv[r] * dk[j][r];
    }
    X = lds.gate.d * X + lds.gate.w[ti] * sum;
#pragma unroll
    for (int i = 32; i >= 1; i >>= 1) X += __shfl_xor(X, i, 64);
    if (lane == 0) lds.x[wave] = X;
  }
  const float2 Gt = lds.gate.g[ti];
  const float e = lds.gate.e[ti], w = lds.gate.w[ti], b = lds.gate.b[ti];
  duv = lds.step[ti];
#pragma unroll
  for (int j = 0; j < NK; ++j) {
    dq[j] *= e;
    y[j] *= e;
    dk[j] *= w;
  }
  // decays and masks
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float x = decay(Gt, lds.gate.g[16 * wave + 4 * g + r]);
    Zd[r] = 4 * g + r <= m ? Zd[r] * x : 0.0f;
    Wd[r] = 4 * g + r < m ? Wd[r] * x : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int o = 16 * j + 4 * g + r;
      const float2 Go = lds.gate.g[o];
      if (j < wave) {
        const float x = decay(Gt, Go);
        Z[j][r] *= x;
        W[j][r] *= x;
      } else {
        const float x = decay(Go, Gt);
        Z[j][r] = o >= ti ? Z[j][r] * x : 0.0f;
        W[j][r] = o > ti ? -lds.gate.b[o] * x * W[j][r] : 0.0f;
      }
    }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    bf16x8 zf[3], wf[3];
    if (2 * h <= wave) {             // rows s at or before t
      const floatx4 z0 = 2 * h < wave ? Z[2 * h] : Zd, w0 = 2 * h < wave ? W[2 * h] : Wd;
      const floatx4 z1 = 2 * h + 1 < wave ? Z[2 * h + 1] : 2 * h + 1 == wave ? Zd : zero;
      const floatx4 w1 = 2 * h + 1 < wave ? W[2 * h + 1] : 2 * h + 1 == wave ? Wd : zero;
      frag_pair(z0, z1, zf);
      frag_pair(w0, w1, wf);
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        bf16x8 f[NP];
        pair_frag_t<NP, DK>(lds.b.k[0], h, j, f);
        mma<NP, 3>(f, zf, dq[j]);
        mma<NP, 3>(f, wf, y[j]);
      }
    }
    if (2 * h + 1 >= wave) {         // rows at or behind it
      const floatx4 z0 = 2 * h >= wave ? Z[2 * h] : zero, w0 = 2 * h >= wave ? W[2 * h] : zero;
      frag_pair(z0, Z[2 * h + 1], zf);
      frag_pair(w0, W[2 * h + 1], wf);
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        bf16x8 f[NP];
        pair_frag_t<NP, DK>(lds.b.q[0], h, j, f);
        mma<NP, 3>(f, zf, dk[j]);
        pair_frag_t<NP, DK>(lds.b.k[0], h, j, f);
        mma<NP, 3>(f, wf, dk[j]);
      }
    }
  }
  // dk = R^T u - b y, and the gates' gradients
  // (a token's own sums in float32: q . dq is as wrong as dq, rounded in float32 accumulators; summed in
  // float64, duv too, dlog_a's error goes from 5.7e-7 to 5.4e-7 at 8x12x2048x64 and the call takes up to
  // 1.7% longer.  Sums over tokens are float64.)
  float qdq = 0.0f, yk = 0.0f;
#pragma unroll
  for (int j = 0; j < NK; ++j) {
    const floatx4 qv = row_values<NP>(lds.b.q[0] + at<DK>(ti, 16 * j + 4 * g), C * DK);
    const floatx4 kv = row_values<NP>(lds.b.k[0] + at<DK>(ti, 16 * j + 4 * g), C * DK);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      qdq += qv[r] * dq[j][r];
      yk += kv[r] * y[j][r];
      dk[j][r] -= b * y[j][r];
    }
    if (ti < left) {
      __builtin_nontemporal_store(dq[j], reinterpret_cast<floatx4*>(a.dq + (row + ti) * DK + 16 * j + 4 * g));
      __builtin_nontemporal_store(dk[j], reinterpret_cast<floatx4*>(a.dk + (row + ti) * DK + 16 * j + 4 * g));
    }
  }
  qdq += __shfl_xor(qdq, 16, 64);
  qdq += __shfl_xor(qdq, 32, 64);
  yk += __shfl_xor(yk, 16, 64);
  yk += __shfl_xor(yk, 32, 64);
  if (g == 0 && ti < left) a.dbeta[row + ti] = duv - yk;
  if (!a.dlog_a) return;
  __syncthreads();
  if (g == 0) lds.step[ti] = qdq - b * duv;
  __syncthreads();
  if (wave > 0) return;
  // lane = token 63 - lane: sums from the chunk's end on, begun anew behind a reset
  const int t = C - 1 - lane;
  const double sum = wave_scan((double)lds.step[t]);
  const bool reset = t < left && is_reset(a.log_a[row + t]);
  const unsigned long long resets = __ballot(reset), before = resets & ((1ull << lane) - 1ull);
  const int last = before ? 63 - __builtin_clzll(before) : 0;
  const double cut = __shfl(sum, last, 64);
  const double out = before ? sum - cut : lds.x[0] + lds.x[1] + lds.x[2] + lds.x[3] + sum;
  if (t < left) a.dlog_a[row + t] = reset ? 0.0f : (float)out;
}

// ------------------------------------------------------------------- plans

constexpr int kChunkThreads = 256;      // of prep_kernel and outputs_kernel, a chunk a workgroup
// Walkers of a workgroup.
constexpr int walkers(int nv) { return nv >= 64 ? 4 : nv / 16; }

struct Plan {
  long chains, chunks;
  int segs, per;
  size_t T, H, G, U, S, R, starts, moves;      // bytes
  size_t bytes() const { return 2 * T + H + G + U + S + R + 2 * starts + 2 * moves; }
  // (a sequence is cut where the launches it takes more have some 256 workgroups)
  bool fit(int nv) const {
    return solve_fits(chains * chunks) && chains * chunks * kChunkThreads < (1l << 32) &&
           fits(2 * (nv / (16 * walkers(nv))), chains * segs, 64 * (walkers(nv) + kKeyWaves));
  }
};
// Walkers' workgroups that a compute unit holds.
template <typename T>
int held_of(int dk) {
  return held(dk == 16 ? sizeof(KeyLds<T, 16>) : dk == 32 ? sizeof(KeyLds<T, 32>)
              : dk == 64 ? sizeof(KeyLds<T, 64>) : sizeof(KeyLds<T, 128>));
}
Plan plan_of(const DeltaBwdArgs& a) {
  Plan p;
  p.chains = (long)a.batch * a.heads;
  p.chunks = ((long)a.seqlen + C - 1) / C;
  const size_t units = (size_t)p.chains * p.chunks, state = (size_t)a.ndv * a.ndk * 4;
  p.T = units * kT * 16;
  p.H = units * C * a.ndv * 4;
  p.G = units * state;
  p.U = (size_t)p.chains * a.seqlen * a.ndv * 4;
  p.S = units * state;
  p.R = units * state;
  const int room = a.dtype == 0 ? held_of<uint16_t>(a.ndk) : held_of<float>(a.ndk);
  const Launch write{write_blocks(a.ndv + a.ndk) + write_blocks(a.ndv), room};
  const Launch walk{2 * (a.ndv / (16 * walkers(a.ndv))), room};
  cut(p.chunks, p.chains, write, 0, walk, a.ndk, p.segs, p.per);
  p.starts = p.segs > 1 ? (size_t)p.chains * p.segs * state : 0;
  p.moves = p.segs > 1 ? (size_t)p.chains * p.segs * move_bytes(a.ndk) : 0;
  return p;
}

template <class K, class... A>
hipError_t go(K kernel, unsigned grid, int threads, size_t bytes, hipStream_t stream, A... args) {
  const hipError_t e = lds_limit(kernel, bytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), bytes, stream, args...);
  return hipGetLastError();
}

template <typename T>
hipError_t run(const DeltaBwdArgs& a, const Plan& p, hipStream_t stream) {
  char* ws = static_cast<char*>(a.workspace);
  auto take = [&](size_t bytes) {
    char* at = ws;
    ws += bytes;
    return at;
  };
  BwdArgs w{a.q, a.k, a.v, a.beta, a.log_a, a.S0, a.dO, a.dS_L, a.dq, a.dk, a.dv, a.dbeta, a.dlog_a, a.dS0};
  uint4* T_ = reinterpret_cast<uint4*>(take(p.T));
  uint4* Tt = reinterpret_cast<uint4*>(take(p.T));
  w.T = T_;
  w.Tt = Tt;
  w.H = reinterpret_cast<float4*>(take(p.H));
  w.G = reinterpret_cast<float4*>(take(p.G));
  w.S = reinterpret_cast<float*>(take(p.S));
  w.R = reinterpret_cast<float*>(take(p.R));
  w.chains = p.chains;
  w.seqlen = a.seqlen;
  w.nv = a.ndv;
  w.segs = p.segs;
  w.per = p.per;
  w.starts_S = reinterpret_cast<float*>(take(p.starts));
  w.starts_R = reinterpret_cast<float*>(take(p.starts));
  w.moves = reinterpret_cast<uint4*>(take(p.moves));
  w.moves_t = reinterpret_cast<uint4*>(take(p.moves));
  w.U = reinterpret_cast<float*>(take(p.U));
  const SolveArgs s{a.k, a.beta, a.log_a, T_, Tt, p.chains, a.seqlen};
  const hipError_t e = launch_solve(s, a.ndk, a.dtype, stream);
  if (e != hipSuccess) return e;
  const int n = (int)p.chunks;
  const unsigned units = (unsigned)(p.chains * p.chunks);
  return with_dim(a.ndk, [&](auto d) {
    constexpr int DK = decltype(d)::value;
    hipError_t e = go(prep_kernel<T, DK>, units, kChunkThreads, sizeof(PrepLds<T, DK>), stream, w, n);
    if (e != hipSuccess) return e;
    auto walks = [&](auto nd) {
      constexpr int ND = decltype(nd)::value;
      if (p.segs > 1) {
        const int blocks = write_blocks(a.ndv + DK) + write_blocks(a.ndv);
        hipError_t e = go(walks_kernel<T, DK, kWriters, true>, grid_of(blocks, p.chains * p.segs),
                          64 * (kWriters + kKeyWaves), sizeof(KeyLds<T, DK>), stream, w, n);
        if (e != hipSuccess) return e;
        const Joins j{{{a.S0, w.starts_S, w.moves, false}, {a.dS_L, w.starts_R, w.moves_t, true}},
                      p.chains, a.ndv, p.segs};
        if ((e = launch_join<DK>(j, 2, stream)) != hipSuccess) return e;
      }
      return go(walks_kernel<T, DK, ND, false>, grid_of(2 * (a.ndv / (16 * ND)), p.chains * p.segs),
                64 * (ND + kKeyWaves), sizeof(KeyLds<T, DK>), stream, w, n);
    };
    const int nd = walkers(a.ndv);
    e = nd == 4   ? walks(std::integral_constant<int, 4>())
        : nd == 2 ? walks(std::integral_constant<int, 2>())
                  : walks(std::integral_constant<int, 1>());
    if (e != hipSuccess) return e;
    static_assert(sizeof(OutLds<T, DK>) <= 163840, "LDS of a workgroup");
    return go(outputs_kernel<T, DK>, units, kChunkThreads, sizeof(OutLds<T, DK>), stream, w, n);
  });
}

}  // namespace
}  // namespace delta

size_t delta_bwd_workspace_bytes(const DeltaBwdArgs& a) { return delta::plan_of(a).bytes(); }

bool delta_bwd_fits(const DeltaBwdArgs& a) { return delta::plan_of(a).fit(a.ndv); }

hipError_t launch_delta_bwd(const DeltaBwdArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  const delta::Plan p = delta::plan_of(a);
  return a.dtype == 0 ? delta::run<uint16_t>(a, p, stream) : delta::run<float>(a, p, stream);
}

}  // namespace falcon
