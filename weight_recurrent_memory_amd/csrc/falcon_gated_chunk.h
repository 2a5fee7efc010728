// falcon_gated_chunk.h - the chunk kernels of the gated recurrence, forward and
// backward.  One form serves all of them: with three sequences x, y (DX columns) and z,
//   out_t = e_t U y_t + sum_{s<=t} D_ts (x_s . y_t) z_s        (a chunk of 64 tokens)
//   U    <- d U + sum_s w_s z_s x_s^T
// D_ts the decay from s to t, e_t from the chunk's start, w_s to its end, d the whole.
//   forward   o  : x = k,  y = q,  z = v,   U = S
//   backward  dq : x = v,  y = dO, z = k,   U = S^T
//             dk : x = dO, y = v,  z = q,   U = R^T   last token first
//             dv : x = q,  y = k,  z = dO,  U = R     last token first
// with R the gradient of the state behind a token.  Walked last token first, a decay
// from s back to t leaves out a_s and takes in a_t's successors: the sums of log decays
// are exclusive in place of inclusive.
//
// Work.  A workgroup (4 waves) takes one segment of one chain for up to 64 z rows and
// walks its chunks in order; wave w owns rows 16w..16w+15 of the chunk for out, and a part
// of U (16 z rows at 64), which stays in its accumulators over the whole segment.  All
// products are 16x16x32 bf16 MFMA over planes.  The scores are formed as P^T = X Y^T: a
// lane then holds 8 scores of one token y_t, with the x rows taken in such an order that
// these are the 8 k-slots the next product (Z^T P^T) wants, so decays, mask and split
// happen in registers.  A chunk's x, z and U lie in LDS by rows; products over
// tokens read x and z transposed; the next chunk's rows are loaded while this one is computed.
//
// Bounds.  Forward at 64 columns (8x12x2048, bf16, 768 workgroups): 30 us, 141 MB over
// the fabric = 4.7 TB/s, nearly a large copy's rate; per chunk and wave about 490 vector and
// 72 matrix instructions.  At 128 columns (1x4x32771): 60 us of issue, two workgroups on a
// compute unit (72 KB of LDS, 250 registers); blocks of 32 z rows in place of 64 make it
// 103 us a call against 92, the scores being formed twice as often.
// What the layout is for: rows as they come from memory and ds_read_b64_tr_b16 for the
// products over tokens, in place of a second, transposed copy: 40 KB in place of 57 at 64
// columns, three workgroups on a compute unit in place of two (a call 63 -> 56 us); reads
// through buffers that end with the sequence, in place of bounds arithmetic (56 -> 53 us at
// 64 columns, 120 -> 103 at 128).  Tried without gain: two chunks ahead in state_kernel;
// the recurrence over segments inside chunk_kernel's first steps (58 us against 54.6).
#pragma once
#include <type_traits>

#include "falcon_gated.h"

namespace falcon {
namespace gated {

// Of two spans (sp1.writes > 0) or one: the states that segments start from, out of every
// segment's own write (falcon_gated.hip).
hipError_t launch_segments(const float* U0, const Span& sp, const float* U1, const Span& sp1, long chains,
                           long state, hipStream_t stream);

namespace {        // (a kernel's name would be exported from the library)

struct ChunkArgs {
  const void* x;         // [chain][L][DX]
  const void* y;
  const void* z;         // [chain][L][nz]
  const float* log_a;    // [chain][L], or null
  const float* U0;       // [chain][state] where the walk starts, or null
  float* out;            // [chain][L][nz]
  float* U_out;          // [chain][state], or null; may be U0
  // gradients of the gates: the part of out_t . u_t that crosses a token's border,
  // that is without s = t; [block][chain][L], or null
  const void* u;         // [chain][L][nz]
  float* dots;
  long chains;
  int seqlen, nz;
};

template <typename TX, typename TZ, int DX, int DZ>
struct LdsState {
  static constexpr int NPX = planes<TX>(), NPZ = planes<TZ>();
  static constexpr int W = DX < 32 ? 32 : DX;       // k-slots come in 32s: zeros behind 16
  static constexpr int WZ = DZ;
  alignas(16) uint16_t x[NPX][C * W];
  alignas(16) uint16_t z[NPZ][C * DZ];
  alignas(16) float2 g[C];                          // sums of log2 decays, row by row
  alignas(16) float e[C];
  alignas(16) float w[C];
  float d;
  alignas(4) unsigned char bad[4];                  // a wave's state is not finite
};
template <typename TX, typename TZ, int DX, int DZ>
struct Lds : LdsState<TX, TZ, DX, DZ> {
  alignas(16) uint16_t s[3][DZ * LdsState<TX, TZ, DX, DZ>::W];   // U at the chunk's start
};

// The workgroup's U: wave w holds z rows 16 (w % NDT).. and NK tiles of 16 x columns.
// A lane's part of a tile: z row lane % 16, x columns 4 (lane / 16) + 0..3.
template <int DX, int DZ>
struct State {
  static constexpr int NDT = DZ / 16, WPD = 4 / NDT, ND = DX / 16, NK = (ND + WPD - 1) / WPD;
  floatx4 t[NK];
  static __device__ __forceinline__ int row0() { return 16 * ((threadIdx.x >> 6) % NDT); }
  static __device__ __forceinline__ int row() { return row0() + (threadIdx.x & 15); }
  static __device__ __forceinline__ int tile(int j) { return ((threadIdx.x >> 6) / NDT) * NK + j; }
  static __device__ __forceinline__ int col(int j) { return 16 * tile(j) + 4 * ((threadIdx.x & 63) >> 4); }
  static __device__ __forceinline__ bool has(int j) { return WPD * NK == ND ? true : tile(j) < ND; }

  // U: element (z, x) at z * sz + x * sx from the block's first row; null: zero
  __device__ __forceinline__ void load(const float* U, long sz, long sx) {
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      t[j] = floatx4{0.f, 0.f, 0.f, 0.f};
      if (!U || !has(j)) continue;
      const float* p = U + row() * sz + col(j) * sx;
      if (sx == 1) t[j] = *reinterpret_cast<const floatx4*>(p);
      else t[j] = floatx4{p[0], p[sx], p[2 * sx], p[3 * sx]};
    }
  }
  __device__ __forceinline__ void store(float* U, long sz, long sx) const {
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      if (!has(j)) continue;
      float* p = U + row() * sz + col(j) * sx;
      if (sx == 1) {
        *reinterpret_cast<floatx4*>(p) = t[j];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i * sx] = t[j][i];
      }
    }
  }
  // (by a sum: one that overflows counts as an entry that does)
  __device__ __forceinline__ bool finite() const {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NK; ++j)
      if (has(j)) s += (t[j].x + t[j].y) + (t[j].z + t[j].w);
    return __builtin_isfinite(s);
  }
  template <int W>
  __device__ __forceinline__ void to_planes(uint16_t* s, int stride) const {
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      if (!has(j)) continue;
      uint2 h, m, l;
      split3(t[j].x, t[j].y, h.x, m.x, l.x);
      split3(t[j].z, t[j].w, h.y, m.y, l.y);
      const int i = at<W>(row(), col(j));
      *reinterpret_cast<uint2*>(s + i) = h;
      *reinterpret_cast<uint2*>(s + stride + i) = m;
      *reinterpret_cast<uint2*>(s + 2 * stride + i) = l;
    }
  }
  // U <- d U + sum_s w_s z_s x_s^T
  template <class L>
  __device__ __forceinline__ void update(const L& lds) {
    constexpr int NPX = L::NPX, NPZ = L::NPZ;
    const int g8 = 8 * ((threadIdx.x & 63) >> 4);
    const float d = lds.d;
#pragma unroll
    for (int j = 0; j < NK; ++j) t[j] *= d;
#pragma unroll
    for (int kk = 0; kk < C; kk += 32) {
      bf16x8 z[NPZ], zw[3];
      float v[8], w[8];
      frag_t<NPZ, L::WZ>(lds.z[0], L::WZ * C, kk + g8, row0(), z);
      values<NPZ>(z, v);
      *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(lds.w + kk + g8);
      *reinterpret_cast<float4*>(w + 4) = *reinterpret_cast<const float4*>(lds.w + kk + g8 + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= w[e];
      frag3(v, zw);
      constexpr int J = NK < 4 ? NK : 4;        // tiles at a time
#pragma unroll
      for (int j0 = 0; j0 < NK; j0 += J) {
        if (NK > J) __builtin_amdgcn_sched_barrier(0);
        bf16x8 x[J][NPX];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int tj = has(j0 + j) ? tile(j0 + j) : 0;
          frag_t<NPX, L::W>(lds.x[0], C * L::W, kk + g8, 16 * tj, x[j]);
        }
#pragma unroll
        for (int p = 0; p < NPX; ++p)
#pragma unroll
          for (int q = 0; p + q < 3; ++q)
#pragma unroll
            for (int j = 0; j < J; ++j) t[j0 + j] = mfma16(x[j][p], zw[q], t[j0 + j]);
      }
    }
  }
};

// One wave's sums of a chunk's log decays, and their place in LDS.  The log decays are
// loaded a chunk earlier than they are summed: a wait for this one load would also be a
// wait for every load issued before it.
struct Decays {
  double g, total;
  float raw;
  template <bool REV>
  __device__ __forceinline__ void load(const float* log_a, long t0, long L) {
    const Window w(log_a ? log_a + t0 : nullptr, log_a ? L - t0 : 0, 1, 0);
    raw = __builtin_bit_cast(float, w.load4b(4 * row_at<REV>(threadIdx.x & 63)));
  }
  template <bool REV>
  __device__ __forceinline__ void sum() {
    const double x = log2_decay(raw);
    g = wave_scan(x);
    total = __shfl(g, 63, 64);
    if (REV) g -= x;
  }
  template <class S>
  __device__ __forceinline__ void store(S& lds) const {
    const int lane = threadIdx.x & 63;
    lds.g[lane] = two_floats(g);
    lds.e[lane] = exp2_of(g);
    lds.w[lane] = exp2_of(total - g);
    if (lane == 0) lds.d = exp2_of(total);
  }
};

// A segment in walking order: its chunks' first tokens.
template <bool REV>
struct Walk {
  long t0;
  int n;
  __device__ __forceinline__ Walk(const Span& sp, int step, long L) {
    const long seg = REV ? sp.segs - 1 - step : step;
    t0 = seg * sp.chunks * C;
    const long left = (L - t0 + C - 1) / C;
    n = left < sp.chunks ? (int)left : sp.chunks;
  }
  __device__ __forceinline__ long at(int c) const { return t0 + (long)(REV ? n - 1 - c : c) * C; }
};

// A segment's own write: U from zero.
template <typename TX, typename TZ, int DX, int DZ, bool REV>
__device__ __forceinline__ void state_body(const ChunkArgs& a, const Span& sp, int blk, long unit,
                                           unsigned char* smem) {
  using L = LdsState<TX, TZ, DX, DZ>;
  L& lds = *reinterpret_cast<L*>(smem);
  const long chain = unit / sp.writes;
  const int step = (int)(unit % sp.writes);
  const int wave = threadIdx.x >> 6;
  const long len = a.seqlen;
  const Walk<REV> walk(sp, step, len);
  const TX* x = static_cast<const TX*>(a.x) + chain * len * DX;
  const TZ* z = static_cast<const TZ*>(a.z) + chain * len * a.nz + blk * DZ;
  const float* la = a.log_a ? a.log_a + chain * len : nullptr;

  Stage<TX, DX, REV> sx(DX);
  Stage<TZ, DZ, REV> sz(a.nz);
  State<DX, DZ> st;
  Decays dec;
  double total = 0.0;
  st.load(nullptr, 0, 1);
  dec.load<REV>(la, walk.at(0), len);
  sx.load(Window(x + walk.at(0) * DX, len - walk.at(0), DX, 0));
  sz.load(Window(z + walk.at(0) * a.nz, len - walk.at(0), a.nz, blk * DZ));
  dec.sum<REV>();
  if (walk.n > 1) dec.load<REV>(la, walk.at(1), len);
  for (int c = 0; c < walk.n; ++c) {
    if (c) __syncthreads();
    sx.template store<L::W>(lds.x[0]);
    sz.template store<DZ>(lds.z[0]);
    if (wave == 0) {
      dec.store(lds);
      total += dec.total;
    }
    __syncthreads();
    if (wave == 0) dec.sum<REV>();
    if (c + 2 < walk.n) dec.load<REV>(la, walk.at(c + 2), len);
    if (c + 1 < walk.n) {
      const long n0 = walk.at(c + 1);
      sx.load(Window(x + n0 * DX, len - n0, DX, 0));
      sz.load(Window(z + n0 * a.nz, len - n0, a.nz, blk * DZ));
    }
    st.update(lds);
  }
  st.store(sp.states + ((chain * (sp.writes + 1) + step + 1) * a.nz + (long)blk * DZ) * DX, DX, 1);
  if (threadIdx.x == 0 && blk == 0) sp.decays[unit] = exp2_of(total);
}
template <typename TX, typename TZ, int DX, int DZ, bool REV>
__global__ __launch_bounds__(NT) void state_kernel(ChunkArgs a, Span sp) {
  extern __shared__ __align__(16) unsigned char smem[];
  int blk;
  long unit;
  if (place(a.nz / DZ, a.chains * sp.writes, blk, unit)) state_body<TX, TZ, DX, DZ, REV>(a, sp, blk, unit, smem);
}

// Four values of NP planes in LDS.
template <int NP>
__device__ __forceinline__ floatx4 values4(const uint16_t* p, int stride) {
  floatx4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = NP - 1; i >= 0; --i) {
    Raw4<uint16_t> r;
    r.u = *reinterpret_cast<const uint2*>(p + i * stride);
    x += r.values();
  }
  return x;
}

// Workgroups on a compute unit that chunk_kernel's registers are held to: with bf16
// operands three up to 64 columns and two at 128, with float32 two and one.  (Three at 128
// columns or two there with float32 spill a hundred registers and more.)
template <typename T, int DX>
constexpr int held() { return planes<T>() == 1 ? (DX <= 64 ? 3 : 2) : (DX <= 64 ? 2 : 1); }

// GRAD: U is kept transposed in memory ([x][z], a state's own layout for dq and dk), and
// dots are written.  Returns true (the forward only), and leaves U_out, where walk_again has
// to follow.
template <typename TX, typename TY, typename TZ, int DX, int DZ, bool REV, bool GRAD>
__device__ __forceinline__ bool chunk_body(const ChunkArgs& a, const Span& sp, int blk, long unit,
                                           unsigned char* smem) {
  using L = Lds<TX, TZ, DX, DZ>;
  constexpr int NPX = L::NPX, NPY = planes<TY>(), NPZ = L::NPZ;
  constexpr int W = L::W, NQ = W / 32, NDT = DZ / 16;
  L& lds = *reinterpret_cast<L*>(smem);
  const long chain = unit / sp.segs;
  const int step = (int)(unit % sp.segs);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m = lane & 15, g = lane >> 4;
  const long len = a.seqlen;
  const Walk<REV> walk(sp, step, len);
  const TX* x = static_cast<const TX*>(a.x) + chain * len * DX;
  const TY* y = static_cast<const TY*>(a.y) + chain * len * DX;
  const TZ* z = static_cast<const TZ*>(a.z) + chain * len * a.nz + blk * DZ;
  const TZ* u = GRAD ? static_cast<const TZ*>(a.u) + chain * len * a.nz + blk * DZ : nullptr;
  const float* la = a.log_a ? a.log_a + chain * len : nullptr;
  float* out = a.out + chain * len * a.nz + blk * DZ;
  const long U_sz = GRAD ? 1 : DX, U_sx = GRAD ? a.nz : 1, U_blk = (long)blk * DZ * U_sz;
  const long state = (long)a.nz * DX;

  Stage<TX, DX, REV> sx(DX);
  Stage<TZ, DZ, REV> sz(a.nz);
  State<DX, DZ> st;
  Decays dec;
  const int ti = 16 * wave + m;                 // this lane's row of the chunk
  Row<TY, DX, REV> ry;
  const int u_at = (row_at<REV>(ti) * a.nz + 4 * g) * (int)sizeof(TZ);
  dec.load<REV>(la, walk.at(0), len);
  sx.load(Window(x + walk.at(0) * DX, len - walk.at(0), DX, 0));
  sz.load(Window(z + walk.at(0) * a.nz, len - walk.at(0), a.nz, blk * DZ));
  ry.load(Window(y + walk.at(0) * DX, len - walk.at(0), DX, 0));
  dec.sum<REV>();
  if (walk.n > 1) dec.load<REV>(la, walk.at(1), len);
  if (sp.segs > 1) st.load(sp.states + (chain * (sp.writes + 1) + step) * state + U_blk, U_sz, U_sx);
  else st.load(a.U0 ? a.U0 + chain * state + U_blk : nullptr, U_sz, U_sx);
  if (DX < W) {      // k-slots behind the last column
    for (int i = threadIdx.x; i < NPX * C * W / 8; i += NT) reinterpret_cast<uint4*>(lds.x[0])[i] = uint4{0u, 0u, 0u, 0u};
    for (int i = threadIdx.x; i < 3 * DZ * W / 8; i += NT) reinterpret_cast<uint4*>(lds.s[0])[i] = uint4{0u, 0u, 0u, 0u};
    __syncthreads();
  }

  for (int c = 0; c < walk.n; ++c) {
    if (c) __syncthreads();
    sx.template store<W>(lds.x[0]);
    sz.template store<DZ>(lds.z[0]);
    st.template to_planes<W>(lds.s[0], DZ * W);
    if (wave == 0) dec.store(lds);
    bf16x8 yf[NQ][NPY];
    ry.frags(yf);
    __syncthreads();
    const long t = token<REV>(walk.at(c), ti);
    // (loads come back in order: the one needed first is issued first)
    Raw4<TZ> ru[NDT];
    if (GRAD) {
      const Window w(u + walk.at(c) * a.nz, len - walk.at(c), a.nz, blk * DZ);
#pragma unroll
      for (int d = 0; d < NDT; ++d) ru[d].load(w, u_at + 16 * d * (int)sizeof(TZ));
    }
    if (wave == 0) dec.sum<REV>();
    if (c + 2 < walk.n) dec.load<REV>(la, walk.at(c + 2), len);
    if (c + 1 < walk.n) {
      const long n0 = walk.at(c + 1);
      sx.load(Window(x + n0 * DX, len - n0, DX, 0));
      sz.load(Window(z + n0 * a.nz, len - n0, a.nz, blk * DZ));
      ry.load(Window(y + n0 * DX, len - n0, DX, 0));
    }

    // out^T: z rows x this wave's 16 tokens; first U's part
    floatx4 acc[NDT];
#pragma unroll
    for (int i = 0; i < NDT; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      if (NQ > 2) __builtin_amdgcn_sched_barrier(0);
      bf16x8 s[NDT][3];
#pragma unroll
      for (int d = 0; d < NDT; ++d) frag<3, W>(lds.s[0], DZ * W, 16 * d + m, 32 * i + 8 * g, s[d]);
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int r = 0; r < NPY; ++r)
          if (p + r < 3) {
#pragma unroll
            for (int d = 0; d < NDT; ++d) acc[d] = mfma16(s[d][p], yf[i][r], acc[d]);
          }
    }
    const float e = lds.e[ti];
    const float2 Gt = lds.g[ti];
#pragma unroll
    for (int d = 0; d < NDT; ++d) acc[d] *= e;
    // then the chunk's own tokens, 32 at a time; none behind the wave's last row
    float same = 0.0f;                          // x_t . y_t, where this lane holds it
#pragma unroll
    for (int kk = 0; kk < C; kk += 32) {
      if (kk > 16 * wave + 15) break;
      __builtin_amdgcn_sched_barrier(0);        // (keeps the reads of a part in that part: registers)
      float v[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // row m of this tile: chunk row kk + 8 (m / 4) + 4 j + m % 4
        floatx4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          bf16x8 xf[NPX];
          frag<NPX, W>(lds.x[0], C * W, kk + 8 * (m >> 2) + 4 * j + (m & 3), 32 * i + 8 * g, xf);
          mma<NPX, NPY>(xf, yf[i], p);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int s = kk + 8 * g + 4 * j + r;
          const float dcy = decay(Gt, lds.g[s]);
          if (GRAD) {                           // s = t is added behind the dots
            v[4 * j + r] = s < ti ? p[r] * dcy : 0.0f;
            same = s == ti ? p[r] : same;
          } else {
            // (walked backward too a token's own term has no decay: dcy = 1)
            v[4 * j + r] = s <= ti ? p[r] * dcy : 0.0f;
          }
        }
      }
      bf16x8 pf[3];
      frag3(v, pf);
      bf16x8 zf[NDT][NPZ];
#pragma unroll
      for (int d = 0; d < NDT; ++d) frag_t<NPZ, DZ>(lds.z[0], DZ * C, kk + 8 * g, 16 * d, zf[d]);
#pragma unroll
      for (int p = 0; p < NPZ; ++p)
#pragma unroll
        for (int r = 0; p + r < 3; ++r)
#pragma unroll
          for (int d = 0; d < NDT; ++d) acc[d] = mfma16(zf[d][p], pf[r], acc[d]);
    }
    if (GRAD) {
      // one of the four lanes of a row holds x_t . y_t, the others 0
      same += __shfl_xor(same, 16, 64);
      same += __shfl_xor(same, 32, 64);
      float dot = 0.0f;
#pragma unroll
      for (int d = 0; d < NDT; ++d) {
        const floatx4 uv = ru[d].values();
        const floatx4 zv = values4<NPZ>(lds.z[0] + at<DZ>(ti, 16 * d + 4 * g), DZ * C);
        dot += acc[d].x * uv.x + acc[d].y * uv.y + acc[d].z * uv.z + acc[d].w * uv.w;
        acc[d] += same * zv;
      }
      dot += __shfl_xor(dot, 16, 64);
      dot += __shfl_xor(dot, 32, 64);
      if (a.dots && g == 0 && t < len) a.dots[(blk * a.chains + chain) * len + t] = dot;
    }
    if (t < len) {
#pragma unroll
      for (int d = 0; d < NDT; ++d)
        __builtin_nontemporal_store(acc[d], reinterpret_cast<floatx4*>(out + t * a.nz + 16 * d + 4 * g));
    }
    st.update(lds);
  }
  if (!REV && !GRAD) {
    // a barrier and a sum of the state, once a segment: 0-1.3% of a call (1x4x32771x128 89.9
    // and 91.2 us, 8x12x2048x64 within noise)
    const bool bad = __any(!st.finite());
    if (lane == 0) lds.bad[wave] = bad;
    __syncthreads();
    if (__builtin_expect(*reinterpret_cast<const unsigned*>(lds.bad) != 0, 0)) return true;
  }
  if (a.U_out && step == sp.segs - 1) st.store(a.U_out + chain * state + U_blk, U_sz, U_sx);
  return false;
}

// The forward's outputs that are not finite formed anew, by the recurrence itself, one token
// at a time.  The products over a chunk's tokens multiply the tokens that a mask leaves out
// with 0, and 0 * NaN is NaN: a NaN or an infinity in v would reach every output of its chunk,
// also of earlier tokens.  The walk's state behind it is not finite either, up to the walk's
// end, which is where it is looked for.  A row of the state lies on 256 / DZ lanes.  Only where
// inputs, or a state that has overflowed, leave no finite state: a call with a NaN in every
// chain takes 396 us in place of 56 (8x12x2048x64), 1039 in place of 94 (1x4x32771x128).
template <typename T, int DX, int DZ>
__device__ __forceinline__ void walk_again(const ChunkArgs& a, const Span& sp, int blk, long unit) {
  constexpr int TPR = NT / DZ, N = DX / TPR;           // 4 to 16 lanes a row, of 1 to 32 columns
  const long chain = unit / sp.segs, len = a.seqlen, state = (long)a.nz * DX;
  const int step = (int)(unit % sp.segs);
  const Walk<false> walk(sp, step, len);
  const long end = walk.t0 + (long)walk.n * C < len ? walk.t0 + (long)walk.n * C : len;
  const int row = blk * DZ + (int)threadIdx.x / TPR, c0 = ((int)threadIdx.x % TPR) * N;
  const long at = (long)row * DX + c0;
  const T* k = static_cast<const T*>(a.x) + chain * len * DX + c0;
  const T* q = static_cast<const T*>(a.y) + chain * len * DX + c0;
  const T* v = static_cast<const T*>(a.z) + chain * len * a.nz + row;
  const float* la = a.log_a ? a.log_a + chain * len : nullptr;
  float* out = a.out + chain * len * a.nz + row;
  const float* S0 = sp.segs > 1 ? sp.states + (chain * (sp.writes + 1) + step) * state
                                : a.U0 ? a.U0 + chain * state : nullptr;
  float S[N];
#pragma unroll
  for (int j = 0; j < N; ++j) S[j] = S0 ? S0[at + j] : 0.0f;
  for (long t = walk.t0; t < end; ++t) {
    const float d = la ? exp2_of(log2_decay(la[t])) : 1.0f, vt = ld_in(v, t * a.nz);
    float o = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      S[j] = d * S[j] + vt * ld_in(k, t * DX + j);
      o += S[j] * ld_in(q, t * DX + j);
    }
    o = group_sum<TPR>(o);
    if (c0 == 0 && !__builtin_isfinite(out[t * a.nz])) out[t * a.nz] = o;
  }
  if (a.U_out && step == sp.segs - 1) {
#pragma unroll
    for (int j = 0; j < N; ++j) a.U_out[chain * state + at + j] = S[j];
  }
}

struct ChunkCall {
  ChunkArgs a;
  Span sp;
};
// The running kernel's arguments read anew: what only a rare path needs is not held in
// registers up to it (held, it spilled scalar registers: 2-4% of a call).
__device__ __forceinline__ ChunkCall call_again() {
  unsigned long at = (unsigned long)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  struct { unsigned w[sizeof(ChunkCall) / 4]; } words;
#pragma unroll
  for (unsigned i = 0; i < sizeof(ChunkCall) / 4; ++i)
    words.w[i] = ((const __attribute__((address_space(4))) unsigned*)at)[i];
  return __builtin_bit_cast(ChunkCall, words);
}
template <typename T, int DX, int DZ>
__global__ __launch_bounds__(NT, (held<T, DX>())) void chunk_kernel(ChunkCall call) {
  extern __shared__ __align__(16) unsigned char smem[];
  int blk;
  long unit;
  if (!place(call.a.nz / DZ, call.a.chains * call.sp.segs, blk, unit)) return;
  if (chunk_body<T, T, T, DX, DZ, false, false>(call.a, call.sp, blk, unit, smem)) {
    const ChunkCall c = call_again();
    place(c.a.nz / DZ, c.a.chains * c.sp.segs, blk, unit);
    walk_again<T, DX, DZ>(c.a, c.sp, blk, unit);
  }
}

// A kernel with more than 64 KB of LDS has to be told so (about a microsecond a call;
// nothing is kept here).
template <class K>
hipError_t lds_limit(K kernel, size_t bytes) {
  if (bytes <= 65536) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename TX, typename TZ, int DX, int DZ, bool REV>
hipError_t go_state(const ChunkArgs& a, const Span& sp, hipStream_t stream) {
  constexpr size_t bytes = sizeof(LdsState<TX, TZ, DX, DZ>);
  auto kernel = state_kernel<TX, TZ, DX, DZ, REV>;
  const hipError_t e = lds_limit(kernel, bytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(grid_of(a.nz / DZ, a.chains * sp.writes)), dim3(NT), bytes, stream, a, sp);
  return hipGetLastError();
}
template <typename T, int DX, int DZ>
hipError_t go_chunk(const ChunkArgs& a, const Span& sp, hipStream_t stream) {
  constexpr size_t bytes = sizeof(Lds<T, T, DX, DZ>);
  auto kernel = chunk_kernel<T, DX, DZ>;
  const hipError_t e = lds_limit(kernel, bytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(grid_of(a.nz / DZ, a.chains * sp.segs)), dim3(NT), bytes, stream,
                     ChunkCall{a, sp});
  return hipGetLastError();
}

// f(size, rows) as constants for dx columns and blocks of `block` z rows.
template <class F>
hipError_t with_sizes(int dx, int block, F&& f) {
  auto rows = [&](auto d) {
    switch (block) {
      case 16: return f(d, std::integral_constant<int, 16>());
      case 32: return f(d, std::integral_constant<int, 32>());
      case 64: return f(d, std::integral_constant<int, 64>());
    }
    return hipErrorInvalidValue;
  };
  switch (dx) {
    case 16: return rows(std::integral_constant<int, 16>());
    case 32: return rows(std::integral_constant<int, 32>());
    case 64: return rows(std::integral_constant<int, 64>());
    case 128: return rows(std::integral_constant<int, 128>());
  }
  return hipErrorInvalidValue;
}

// The states that segments start from: every segment's own write, then the recurrence
// over segments.
template <typename TX, typename TZ, bool REV>
hipError_t launch_states(const ChunkArgs& a, int dx, int block, const Span& sp, hipStream_t stream) {
  if (sp.writes == 0) return hipSuccess;
  const hipError_t e = with_sizes(dx, block, [&](auto d, auto r) {
    return go_state<TX, TZ, decltype(d)::value, decltype(r)::value, REV>(a, sp, stream);
  });
  return e != hipSuccess ? e : launch_segments(a.U0, sp, nullptr, Span{}, a.chains, (long)a.nz * dx, stream);
}

// Floats of a span's workspace.
inline size_t span_floats(const Span& sp, long chains, long state) {
  return sp.writes ? (size_t)chains * ((size_t)(sp.writes + 1) * state + sp.writes) : 0;
}
// Takes them from p, which moves behind (to a multiple of 16 bytes).
inline void place_span(Span& sp, long chains, long state, float*& p) {
  if (sp.writes == 0) return;
  sp.states = p;
  sp.decays = p + (size_t)chains * (sp.writes + 1) * state;
  p += (span_floats(sp, chains, state) + 3) / 4 * 4;
}
inline size_t span_bytes(const Span& sp, long chains, long state) {
  return (span_floats(sp, chains, state) + 3) / 4 * 16;
}

}  // namespace
}  // namespace gated
}  // namespace falcon
