// falcon_delta_walk.h - the wave that walks a sequence's chunks in order with 16 value rows of
// the gated delta rule's state, the waves that bring keys and gates to LDS for it, and the
// segments of a long sequence.
//
// The walk S -> X -> U -> S is one chain of dependent products, so its latency counts, not its
// operations: a chunk takes a wave 2.2 us at 64 columns (84 matrix and about 430 vector
// instructions, of which 352 split float32 values into bf16 planes; some 75% of the time is
// issue) and 3.4 us at 128, whatever else the compute unit does.  Value rows do not
// depend on each other: each wave takes 16, and there is no exchange and no barrier inside a
// chunk, one barrier a chunk for keys and gates.
#pragma once
#include "falcon_delta.h"

namespace falcon {
namespace delta {
namespace {        // (a kernel's name would be exported from the library)

// Chunks that K and gates are in LDS before they are used.  Two where there are registers for
// a chunk's first operands behind the chunk before it.
template <typename T, int DK>
constexpr int ahead() { return planes<T>() == 1 && DK <= 64 ? 2 : 1; }

template <typename T, int DK>
struct StateLds {
  static constexpr int NP = planes<T>(), NQ = (DK + 31) / 32, R = ahead<T, DK>() + 1;
  alignas(16) uint16_t k[R][NP][C * DK];
  Gates gate[R];
  alignas(16) unsigned char bad[4];
};
// The same with T, for workgroups of walkers alone: one read of T from memory serves them all, and
// the walkers' registers are free of it (each with T in its own: 32 us in place of 26 for the
// gradients' walks at 1x5x4099, 128x64).
template <typename T, int DK>
struct KeyLds : StateLds<T, DK> {
  alignas(16) uint4 t[2][kT];
};

// T's operands as a walker has them: read ahead into registers, or from LDS where they are used.
struct RegT {
  bf16x8 f[kFrags][3];
  __device__ __forceinline__ void load(const uint4* p) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kFrags; ++i)
#pragma unroll
      for (int n = 0; n < 3; ++n) f[i][n] = __builtin_bit_cast(bf16x8, p[(i * 3 + n) * 64 + lane]);
  }
  __device__ __forceinline__ bf16x8 get(int i, int n) const { return f[i][n]; }
};
struct LdsT {
  const uint4* p;
  __device__ __forceinline__ bf16x8 get(int i, int n) const {
    return __builtin_bit_cast(bf16x8, p[(i * 3 + n) * 64 + (threadIdx.x & 63)]);
  }
};

// S^T: 16 value rows, columns of keys in tiles of 16.
template <int DK>
struct StateT {
  static constexpr int NK = DK / 16, NQ = (DK + 31) / 32;
  floatx4 t[NK];
  __device__ __forceinline__ void load(const float* S) {       // rows of the 16, or null
    const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int j = 0; j < NK; ++j)
      t[j] = S ? *reinterpret_cast<const floatx4*>(S + m * DK + 16 * j + 4 * g) : floatx4{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void unit(int row0) {             // rows of the unit matrix
    const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) t[j][r] = row0 + m == 16 * j + 4 * g + r ? 1.0f : 0.0f;
  }
  __device__ __forceinline__ void store(float* S) const {
    const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int j = 0; j < NK; ++j) *reinterpret_cast<floatx4*>(S + m * DK + 16 * j + 4 * g) = t[j];
  }
  __device__ __forceinline__ void frag(int i, bf16x8 (&f)[3]) const {
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    if constexpr (DK == 16) frag_pair(t[0], zero, f);
    else frag_pair(t[2 * i], t[2 * i + 1], f);
  }
  // The 16 unit rows of tile w, walked, as a join's operands: `back`'s rows are these rows, `ahead`'s
  // the columns (either may be null; kMove uint4 each).  A product with the unit matrix exchanges
  // rows and columns of a tile; its three planes' sum is exact.
  static constexpr int kMove = NK * NQ * 3 * 64;
  __device__ __forceinline__ void store_moves(uint4* ahead, uint4* back, int w) const {
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    bf16x8 f[3];
    if (back) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        frag(i, f);
#pragma unroll
        for (int p = 0; p < 3; ++p) back[((w * NQ + i) * 3 + p) * 64 + lane] = __builtin_bit_cast(uint4, f[p]);
      }
    }
    if (!ahead) return;
    uint2 e;                             // bf16 1.0 where slot 4 g + i is column m
    e.x = (4 * g == m ? 0x3F80u : 0u) | (4 * g + 1 == m ? 0x3F800000u : 0u);
    e.y = (4 * g + 2 == m ? 0x3F80u : 0u) | (4 * g + 3 == m ? 0x3F800000u : 0u);
    const bf16x8 unit_matrix = __builtin_bit_cast(bf16x8, uint4{e.x, e.y, 0u, 0u});
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      floatx4 x = zero;
      frag_pair(t[j], zero, f);
#pragma unroll
      for (int p = 0; p < 3; ++p) x = mfma16(f[p], unit_matrix, x);
      uint2 h[3];
      split3(x.x, x.y, h[0].x, h[1].x, h[2].x);
      split3(x.z, x.w, h[0].y, h[1].y, h[2].y);
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        uint4* to = ahead + ((j * NQ + w / 2) * 3 + p) * 64 + lane;
        if (DK == 16) *to = uint4{h[p].x, h[p].y, 0u, 0u};
        else reinterpret_cast<uint2*>(to)[w & 1] = h[p];
      }
    }
  }
  __device__ __forceinline__ bool finite() const {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NK; ++j) s += (t[j].x + t[j].y) + (t[j].z + t[j].w);
    return __builtin_isfinite(s);
  }
};

// The wave that owns 16 value rows: S through the chunks of a segment.
template <typename T, int DK, class TT>
struct Walker {
  static constexpr int NP = planes<T>(), NQ = (DK + 31) / 32, NK = DK / 16;
  StateT<DK> S;
  TT t;
  float v[16];

  // v: the sequence's rows from the chunk's first token on; col: of the 16 rows' first
  __device__ __forceinline__ void load_v(const T* p, long rows, int nv, int col) {
    const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    const Window w(p, rows, nv, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[4 * i + r] = load_one(w, (16 * i + 4 * g + r) * nv + col + m, T());
  }

  static constexpr bool kAhead = ahead<T, DK>() > 1;
  bf16x8 kf[kAhead ? NQ : 1][4][NP];      // K's rows

  __device__ __forceinline__ void load_k_step(const uint16_t* k, int n, bf16x8 (&f)[4][NP]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) pair_frag<NP, DK>(k, 16 * i + (threadIdx.x & 15), n, f[i]);
  }
  __device__ __forceinline__ void load_k(const uint16_t* k) {
    if constexpr (kAhead) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) load_k_step(k, n, kf[n]);
    }
  }

  // One chunk; store(index, plane, fragment) gets S's operands, values(U) U, pairs(n, U) U once
  // tiles 2 n and 2 n + 1 are on their way into S.  load() is called once v and T are used,
  // last() behind everything.
  template <class Load, class Last, class Store, class Values, class Pairs>
  __device__ __forceinline__ void chunk(const uint16_t* k, const Gates& gt, Load&& load, Last&& last, Store&& store,
                                        Values&& values, Pairs&& pairs) {
    const int g = (threadIdx.x & 63) >> 4;
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    // K S^T
    floatx4 x[4] = {zero, zero, zero, zero}, b[4], be[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[i] = four(gt.b + 16 * i + 4 * g);
      be[i] = four(gt.be + 16 * i + 4 * g);
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      bf16x8 s[3];
      S.frag(n, s);
#pragma unroll
      for (int p = 0; p < 3; ++p) store(n, p, s[p]);
      bf16x8(&kn)[4][NP] = kf[kAhead ? n : 0];
      if (!kAhead) load_k_step(k, n, kn);
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int r = 0; p + r < 3; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = mfma16(kn[i][p], s[r], x[i]);
    }
    // X = b v - b e K S^T, then U = T X
    bf16x8 xf[3];
    floatx4 u[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 2 * j; i < 2 * j + 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[i][r] = b[i][r] * v[4 * i + r] - be[i][r] * x[i][r];
      frag_pair(x[2 * j], x[2 * j + 1], xf);
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int i = 2 * j; i < 4; ++i) {
          const bf16x8 tf = t.get(frag_of(i, j), p);
#pragma unroll
          for (int r = 0; p + r < 3; ++r) u[i] = mfma16(tf, xf[r], u[i]);
        }
    }
    load();
    values(u);
    // S <- d S + (w U)^T K
    bf16x8 f[3];
    floatx4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = four(gt.w + 16 * i + 4 * g);
    const float d = gt.d;
#pragma unroll
    for (int j = 0; j < NK; ++j) S.t[j] *= d;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      frag_pair(u[2 * n] * w[2 * n], u[2 * n + 1] * w[2 * n + 1], f);
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
            for (int j = 0; j < J; ++j) S.t[j0 + j] = mfma16(kt[j][p], f[r], S.t[j0 + j]);
      }
      pairs(n, u);
    }
    last();
  }
};

// K rows of a chunk on their way to LDS, by N waves.
template <typename T, int DK, int NTH>
struct StageK {
  static constexpr int NP = planes<T>(), G = DK / 8, UNITS = C * G, N = (UNITS + NTH - 1) / NTH;
  Raw<T> r[N];
  __device__ __forceinline__ void load(const Window& w, int t) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = t + i * NTH;
      r[i].load(w, UNITS % NTH == 0 || u < UNITS ? 8 * u * (int)sizeof(T) : kNowhere);
    }
  }
  __device__ __forceinline__ void store(uint16_t* k, int t) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = t + i * NTH;
      if (UNITS % NTH != 0 && u >= UNITS) continue;
      uint4 a[NP];
      r[i].split(a);
#pragma unroll
      for (int p = 0; p < NP; ++p) *reinterpret_cast<uint4*>(k + p * C * DK + at<DK>(u / G, 8 * (u % G))) = a[p];
    }
  }
};

// The waves beside the walkers: K and gates, a chunk or two ahead.  REV: last chunk first.
template <typename T, int DK, int NTH, bool REV>
struct Keys {
  static constexpr int D = ahead<T, DK>(), R = D + 1;
  StageK<T, DK, NTH> sk;
  GateLoad gl;
  const T* k;
  const float* la;
  const float* be;
  long left;
  int n, t;
  __device__ __forceinline__ void load(int c) {
    const long at = (long)(REV ? n - 1 - c : c) * C;
    sk.load(Window(k + at * DK, left - at, DK, 0), t);
    gl.load(la, be, at, left);
  }
  // to the place of chunk `to`
  __device__ __forceinline__ void store(StateLds<T, DK>& lds, int to) const {
    sk.store(lds.k[to % R][0], t);
    if (t < 64) gl.store(lds.gate[to % R]);
  }
  // t: thread of the NTH; k, la, be and `left` tokens from the walk's first token on
  __device__ __forceinline__ Keys(StateLds<T, DK>& lds, const T* k_, const float* la_, const float* be_, long left_,
                                  int n_, int t_)
      : k(k_), la(la_), be(be_), left(left_), n(n_), t(t_) {
#pragma unroll
    for (int c = 0; c < D; ++c) {
      if (c >= n) break;
      load(c);
      store(lds, c);
    }
  }
};

constexpr int kKeyWaves = 2;             // of a workgroup without outputs: these bring T, too
// T on its way to LDS.
template <int NTH>
struct StageT {
  static constexpr int N = kT / NTH;
  static_assert(kT % NTH == 0, "whole units of T a thread");
  uint4_t r[N];            // (a plain vector: an array of HIP's own type stays in memory)
  __device__ __forceinline__ void load(const uint4* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = *reinterpret_cast<const uint4_t*>(p + i * NTH);
  }
  __device__ __forceinline__ void store(uint4* p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<uint4_t*>(p + i * NTH) = r[i];
  }
};
// What a step stores was loaded in the step before it, so that a load has a chunk's time to come
// back (loaded and stored in one step the walkers waited for it: 136 us in place of 127 for the
// gradients' walks at 8x12x2048x64).  Behind
// the last chunk it is loaded and stored once more, to places that are not read: no branches.
// T_: the walk's first chunk's in memory (REV: the last one walked)
template <typename T, int DK, bool REV>
__device__ __forceinline__ void keys_only(KeyLds<T, DK>& lds, const T* k, const float* la, const float* be,
                                          const uint4* T_, long left, int n, int t) {
  StageT<64 * kKeyWaves> st;
  T_ += t;
  st.load(T_ + (long)(REV ? n - 1 : 0) * kT);
  Keys<T, DK, 64 * kKeyWaves, REV> keys(lds, k, la, be, left, n, t);
  constexpr int D = keys.D;
  st.store(lds.t[0] + t);
  const int last = n - 1;
  {
    const int next = n > 1 ? 1 : 0;
    st.load(T_ + (long)(REV ? last - next : next) * kT);
  }
  keys.load(D < n ? D : last);
  for (int c = 0; c < n; ++c) {
    __syncthreads();
    st.store(lds.t[(c + 1) & 1] + t);
    keys.store(lds, c + D);
    __builtin_amdgcn_sched_barrier(0);
    const int next = c + 2 < n ? c + 2 : last;
    st.load(T_ + (long)(REV ? last - next : next) * kT);
    keys.load(c + D + 1 < n ? c + D + 1 : last);
    __builtin_amdgcn_sched_barrier(0);
  }
  __syncthreads();
}

// ------------------------------------------------------------- segments
// A long sequence of few chains is cut into segments that are walked side by side.  The rule
// is affine in S, S -> S M + N with M (dk x dk) and N of the segment alone: a first launch
// walks every segment from zero (N) and from unit rows (M), a second joins them in order, the
// main walk then starts each segment from its state.  R -> R M^T + N' for the gradient's.

// State waves of the first launch's workgroups, one for each SIMD of a compute unit whatever dv
// is, and its workgroups for so many value and unit rows of a segment.
constexpr int kWriters = 4;
__host__ __device__ constexpr int write_blocks(int rows) { return (rows + 16 * kWriters - 1) / (16 * kWriters); }

// A launch's workgroups for one segment, which lie on one of the GPU's 8 XCDs (place), of 32 compute
// units, and how many of them a compute unit holds (by LDS).
struct Launch {
  int blocks, held;
};
constexpr int held(size_t lds) { return lds <= 163840 / 2 ? 2 : 1; }
inline long rounds(const Launch& l, long segments) {
  const long all = (segments + 7) / 8 * l.blocks, room = 32 * l.held;
  return (all + room - 1) / room;
}

// Segments of two chunks at least, 256 workgroups of the first launch aimed at (one a compute unit, a
// walker a SIMD; `unwritten` segments of a chain are not in it).  A chain is cut where two walks of a
// segment, each in its rounds, are at least kGain chunks shorter than one of the whole, which is what
// the two launches more cost.  Measured, us of a call cut and whole, forward and gradients:
// 1x16x4096x64 66 and 137, 153 and 235; 1x8x2048x64 45 and 76, 70 and 120; 1x3x3000x32 34 and 88, 52
// and 125; 1x20x2048x128 98 and 113; 1x12x4096x128 the gradients 292 and 364; 1x1x768x128 (8 chunks
// shorter) 42 and 50, 81 and 88; 1x2x640x64 (6) 31 and 33, 51 and 58; but 1x27x704x64 (5) 40 and 38;
// 1x4x512x128 (4) 40 and 39, 82 and 79; 1x20x1024x128 (4) 66 and 65; 1x20x640x128 (2) 56 and 48.
// With 512 slots 1x16x4096x64 takes 76 and 163.  Narrow values: 1x9x4096, 128x16 81 and 186, 141 and
// 218; 1x28x4096, 128x32 fp32 237 and 308.  Two rounds, fp32: of the main walk 1x20x2048x128 184 and
// 160; of the first launch 1x28x4096, 64x16 the gradients 259 and 245, 64x32 286 and 269.  At 128 columns
// a second round of the first launch, which stores no states, takes 4.0 us a chunk against 6.0 of the
// main walk's, and is not counted: 1x14x4096x128 the gradients 522 and 551.
constexpr long kGain = 6, kSlots = 256;
inline void cut(long chunks, long chains, const Launch& write, int unwritten, const Launch& walk, int dk, int& segs,
                int& per) {
  segs = 1;
  per = (int)chunks;
  long n = kSlots / (chains * write.blocks);
  if (n > chunks / 2) n = chunks / 2;
  if (n < 2) return;
  const long each = (chunks + n - 1) / n;
  n = (chunks + each - 1) / each;
  const long first = dk < 128 ? rounds(write, chains * (n - unwritten)) : 1;
  if (each * (first + rounds(walk, chains * n)) + kGain > chunks * rounds(walk, chains)) return;
  per = (int)each;
  segs = (int)n;
}

// A wave behind the last of these rows: the walkers' barriers.
__device__ __forceinline__ void idle(int chunks) {
  for (int c = 0; c <= chunks; ++c) __syncthreads();
}

// Bytes of a segment's matrix as a join's operands (StateT::kMove).
inline size_t move_bytes(int dk) { return (size_t)(dk / 16) * ((dk + 31) / 32) * 3 * 64 * 16; }

struct Join {
  const float* S0;         // or null
  float* starts;           // [chain][segs][dv][dk]: slot j + 1 step j's own write, then slot j what step j starts from
  const uint4* moves;      // [chain][segs][StateT::kMove], planes (whose splitting took half of a join)
  bool reverse;            // the first step is the last segment
};
struct Joins {
  Join j[2];
  long chains;
  int nv, segs;
};

// start of step j + 1 = (start of j) M_j + write of j, in place.  A workgroup takes 16 value rows of
// a chain, a wave 16 columns of the result; operands of two steps are on their way.
template <int DK>
__global__ __launch_bounds__(4 * DK) void join_kernel(Joins all) {
  constexpr int NQ = (DK + 31) / 32;
  __shared__ __align__(16) uint2 s[2][NQ][3][64][2];
  const Join a = all.j[blockIdx.y];
  const int wave = wave_id(), lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int blocks = all.nv / 16, steps = all.segs - 1;
  int blk;
  long chain;
  if (!place(blocks, all.chains, blk, chain)) return;      // (a chain's blocks read its moves in one XCD's L2)
  const long state = (long)all.nv * DK, row = blk * 16 + m;
  const long at = row * DK + 16 * wave + 4 * g;
  float* starts = a.starts + chain * all.segs * state + at;
  constexpr long kMove = StateT<DK>::kMove;
  const uint4* moves = a.moves + (chain * all.segs + (a.reverse ? steps : 0)) * kMove + wave * NQ * 3 * 64 + lane;
  const long stride = a.reverse ? -kMove : kMove;
  const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
  floatx4 x = a.S0 ? *reinterpret_cast<const floatx4*>(a.S0 + chain * state + at) : zero;
  *reinterpret_cast<floatx4*>(starts) = x;
  if (DK == 16) {
    for (int i = threadIdx.x; i < 2 * 3 * 64; i += 64) (&s[0][0][0][0][0])[2 * i + 1] = uint2{0u, 0u};
  }
  struct Step {
    uint4_t f[NQ][3];
    floatx4 w;
  } ahead[2];
  auto fetch = [&](Step& o, int j) {
    if (j >= steps) j = steps - 1;       // (no branch: one would wait for what is on its way)
    o.w = *reinterpret_cast<const floatx4*>(starts + (j + 1) * state);
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int p = 0; p < 3; ++p) o.f[i][p] = *reinterpret_cast<const uint4_t*>(moves + j * stride + (i * 3 + p) * 64);
  };
  auto step = [&](Step& o, int j, int buf) {
    uint2 h, mi, l;
    split3(x.x, x.y, h.x, mi.x, l.x);
    split3(x.z, x.w, h.y, mi.y, l.y);
    uint2 (*to)[64][2] = s[buf][wave / 2];
    to[0][lane][wave & 1] = h;
    to[1][lane][wave & 1] = mi;
    to[2][lane][wave & 1] = l;
    bf16x8 f[NQ][3];
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int p = 0; p < 3; ++p) f[i][p] = __builtin_bit_cast(bf16x8, o.f[i][p]);
    x = o.w;
    fetch(o, j + 2);
    __syncthreads();
    floatx4 y = zero;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      bf16x8 b[3];
#pragma unroll
      for (int p = 0; p < 3; ++p) b[p] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(s[buf][i][p][lane]));
      if (i & 1) mma<3, 3>(f[i], b, y);
      else mma<3, 3>(f[i], b, x);
    }
    x += y;
    *reinterpret_cast<floatx4*>(starts + (j + 1) * state) = x;
  };
  fetch(ahead[0], 0);
  fetch(ahead[1], 1);
  for (int j = 0; j < steps; j += 2) {
    step(ahead[0], j, 0);
    if (j + 1 < steps) step(ahead[1], j + 1, 1);
  }
}
template <int DK>
hipError_t launch_join(const Joins& j, int directions, hipStream_t stream) {
  hipLaunchKernelGGL((join_kernel<DK>), dim3(grid_of(j.nv / 16, j.chains), directions), dim3(4 * DK), 0, stream, j);
  return hipGetLastError();
}

}  // namespace
}  // namespace delta
}  // namespace falcon
