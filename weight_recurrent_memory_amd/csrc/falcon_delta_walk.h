// falcon_delta_walk.h - the wave that walks a sequence's chunks in order with 16 value rows of
// the gated delta rule's state, and the waves that bring keys and gates to LDS for it.
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
  __device__ __forceinline__ void store_transposed(float* S, int row0) const {
    const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[(16 * j + 4 * g + r) * DK + row0 + m] = t[j][r];
  }
  __device__ __forceinline__ void frag(int i, bf16x8 (&f)[3]) const {
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    if constexpr (DK == 16) frag_pair(t[0], zero, f);
    else frag_pair(t[2 * i], t[2 * i + 1], f);
  }
  __device__ __forceinline__ bool finite() const {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NK; ++j) s += (t[j].x + t[j].y) + (t[j].z + t[j].w);
    return __builtin_isfinite(s);
  }
};

// The wave that owns 16 value rows: S through the chunks of a segment.
template <typename T, int DK>
struct Walker {
  static constexpr int NP = planes<T>(), NQ = (DK + 31) / 32, NK = DK / 16;
  StateT<DK> S;
  bf16x8 T_[kFrags][3];
  float v[16];

  __device__ __forceinline__ void load_T(const uint4* p) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
#pragma unroll
      for (int n = 0; n < 3; ++n) T_[f][n] = __builtin_bit_cast(bf16x8, p[(f * 3 + n) * 64 + lane]);
  }
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

  // One chunk; store(which, index, plane, fragment) gets S's and (FRAGS) U's operands,
  // values(U) U itself.  load() is called once v and T are used, last() behind everything.
  template <bool FRAGS, class Load, class Last, class Store, class Values>
  __device__ __forceinline__ void chunk(const uint16_t* k, const Gates& gt, Load&& load, Last&& last, Store&& store,
                                        Values&& values) {
    const int g = (threadIdx.x & 63) >> 4;
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    // K S^T
    floatx4 x[4] = {zero, zero, zero, zero}, b[4], be[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[i] = *reinterpret_cast<const floatx4*>(gt.b + 16 * i + 4 * g);
      be[i] = *reinterpret_cast<const floatx4*>(gt.be + 16 * i + 4 * g);
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      bf16x8 s[3];
      S.frag(n, s);
#pragma unroll
      for (int p = 0; p < 3; ++p) store(0, n, p, s[p]);
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
        for (int r = 0; p + r < 3; ++r)
#pragma unroll
          for (int i = 2 * j; i < 4; ++i) u[i] = mfma16(T_[frag_of(i, j)][p], xf[r], u[i]);
    }
    load();
    values(u);
    // S <- d S + (w U)^T K
    bf16x8 f[3];
    floatx4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const floatx4*>(gt.w + 16 * i + 4 * g);
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
      if constexpr (FRAGS) {
        frag_pair(u[2 * n], u[2 * n + 1], f);
#pragma unroll
        for (int p = 0; p < 3; ++p) store(1, n, p, f[p]);
      }
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
  __device__ __forceinline__ void store(StateLds<T, DK>& lds, int c) const {
    sk.store(lds.k[c % R][0], t);
    if (t < 64) gl.store(lds.gate[c % R]);
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

constexpr int kKeyWaves = 2;             // of a workgroup without outputs
template <typename T, int DK, bool REV>
__device__ __forceinline__ void keys_only(StateLds<T, DK>& lds, const T* k, const float* la, const float* be,
                                          long left, int n, int t) {
  Keys<T, DK, 64 * kKeyWaves, REV> keys(lds, k, la, be, left, n, t);
  for (int c = 0; c < n; ++c) {
    __syncthreads();
    if (c + keys.D < n) {
      keys.load(c + keys.D);
      keys.store(lds, c + keys.D);
    }
  }
  __syncthreads();
}

}  // namespace
}  // namespace delta
}  // namespace falcon
