// falcon_gated.h - shared pieces of the gated recurrence's chunk kernels: operands as
// planes of bf16, their place in LDS, the sums of log decays.
//
// Planes.  An exact bf16 operand is one plane.  A float32 operand x is three: h =
// bf16(x), m = bf16(x - h), l = bf16(x - h - m), whose sum is x to 24 bits.  A product
// runs the plane pairs (i, j) with i + j < 3, so what is left out is 2^-24 of it: the
// matrix cores' bf16 rate (16 times the float32 one) at float32's precision, three
// passes with one float32 operand and six with two.
//
// Decays.  G_t = sum of log2 a over the chunk up to t, in float64: the decay from s to
// t is 2^(G_t - G_s), one subtraction and one v_exp.  In float32 a reset (a log decay
// of -1000) would leave the differences behind it wrong by 2^-24 of 1000.  A decay is
// never divided by.
#pragma once
#include "falcon_device.h"
#include "falcon_launch.h"

namespace falcon {
namespace gated {

constexpr int C = 64;          // tokens of a chunk
constexpr int NT = 256;        // threads of a workgroup, 16 tokens of a chunk a wave

template <typename T>
constexpr int planes() { return sizeof(T) == 2 ? 1 : 3; }

// Element offset of (row, col) in a plane of rows of W (32, 64 or 128) bf16: groups of
// 8 elements (16 bytes) are XORed with bits of the row, so that the 16-byte reads of 8
// consecutive rows, of rows 0-3 and 8-11 together, and the transposing writes to rows 8
// apart each fall into different banks.
template <int W>
__device__ __forceinline__ int at(int row, int col) {
  const int x = row >> 3;
  const int f = (row & 7) ^ (((x & 1) << 2) | (x & 2) | ((x >> 2) & 1));
  return row * W + (((col >> 3) ^ (f & (W / 8 - 1))) << 3) + (col & 7);
}

// Three planes of a pair of floats, packed.
__device__ __forceinline__ void split3(float a, float b, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = pack_bf16x2(a, b);
  const float ra = a - __uint_as_float(h << 16), rb = b - __uint_as_float(h & 0xFFFF0000u);
  m = pack_bf16x2(ra, rb);
  l = pack_bf16x2(ra - __uint_as_float(m << 16), rb - __uint_as_float(m & 0xFFFF0000u));
}
__device__ __forceinline__ void frag3(const float (&x)[8], bf16x8 (&f)[3]) {
  uint4 h, m, l;
  split3(x[0], x[1], h.x, m.x, l.x);
  split3(x[2], x[3], h.y, m.y, l.y);
  split3(x[4], x[5], h.z, m.z, l.z);
  split3(x[6], x[7], h.w, m.w, l.w);
  f[0] = __builtin_bit_cast(bf16x8, h);
  f[1] = __builtin_bit_cast(bf16x8, m);
  f[2] = __builtin_bit_cast(bf16x8, l);
}
// The values a fragment's planes stand for.
template <int NP>
__device__ __forceinline__ void values(const bf16x8 (&f)[NP], float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = (float)f[NP - 1][e];
#pragma unroll
    for (int p = NP - 2; p >= 0; --p) x[e] += (float)f[p][e];
  }
}

// Eight consecutive inputs as they are in memory, and as planes.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  uint4 u;
  __device__ __forceinline__ void load(const uint16_t* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = uint4{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void split(uint4 (&f)[1]) const { f[0] = u; }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = float4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void split(uint4 (&f)[3]) const {
    split3(a.x, a.y, f[0].x, f[1].x, f[2].x);
    split3(a.z, a.w, f[0].y, f[1].y, f[2].y);
    split3(b.x, b.y, f[0].z, f[1].z, f[2].z);
    split3(b.z, b.w, f[0].w, f[1].w, f[2].w);
  }
};

// One MFMA operand fragment (NP planes) from row `row`, columns col..col+7 of planes
// `stride` elements apart.
template <int NP, int W>
__device__ __forceinline__ void frag(const uint16_t* p, int stride, int row, int col,
                                     bf16x8 (&f)[NP]) {
#pragma unroll
  for (int i = 0; i < NP; ++i) f[i] = frag_bf16(p + i * stride + at<W>(row, col));
}

// Token of row `row` of the chunk of tokens t0..t0+63.
template <bool REV>
__device__ __forceinline__ long token(long t0, int row) { return t0 + (REV ? C - 1 - row : row); }

// A chunk's rows of one input on its way to LDS: units of two tokens x 8 columns,
// `units()` of them over the workgroup's threads.
template <typename T, int D>
struct Stage {
  static constexpr int NP = planes<T>();
  static constexpr int G = D / 8, UNITS = (C / 2) * G, N = (UNITS + NT - 1) / NT;
  Raw<T> r[N][2];

  // the 64 tokens from t0 on, rows of `ld` elements (REV: the last token first); tokens
  // from L on are zero
  template <bool REV>
  __device__ __forceinline__ void load(const T* x, long t0, long L, int ld) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = threadIdx.x + i * NT;
      const bool mine = UNITS % NT == 0 || u < UNITS;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const long t = token<REV>(t0, 2 * (u / G) + j);
        if (mine && t < L) r[i][j].load(x + t * ld + 8 * (u % G));
        else r[i][j].zero();
      }
    }
  }
  // to rows[token][column] (W wide, or null) and cols[column][token] (64 wide, or null)
  template <int W>
  __device__ __forceinline__ void store(uint16_t* rows, uint16_t* cols) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = threadIdx.x + i * NT;
      if (UNITS % NT != 0 && u >= UNITS) continue;
      const int s = 2 * (u / G), c = 8 * (u % G);
      uint4 a[NP], b[NP];
      r[i][0].split(a);
      r[i][1].split(b);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        if (rows) {
          *reinterpret_cast<uint4*>(rows + p * C * W + at<W>(s, c)) = a[p];
          *reinterpret_cast<uint4*>(rows + p * C * W + at<W>(s + 1, c)) = b[p];
        }
        if (cols) {
          const uint32_t x[4] = {a[p].x, a[p].y, a[p].z, a[p].w};
          const uint32_t y[4] = {b[p].x, b[p].y, b[p].z, b[p].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // (token s, token s + 1) of column c + e
            const uint32_t lo = e & 1 ? x[e / 2] >> 16 : x[e / 2] & 0xFFFFu;
            const uint32_t hi = e & 1 ? y[e / 2] & 0xFFFF0000u : y[e / 2] << 16;
            *reinterpret_cast<uint32_t*>(cols + p * D * C + at<C>(c + e, s)) = lo | hi;
          }
        }
      }
    }
  }
};

// log2 of the decay of token t (0 from L on and without gates), at least -1000 log2 e.
__device__ __forceinline__ double log2_decay(const float* log_a, long t, long L) {
  float g = log_a && t < L ? log_a[t] : 0.0f;
  g = g < -1000.0f ? -1000.0f : g;
  return (double)g * 1.4426950408889634;
}
// Inclusive sum over the lanes of a wave, first lane first.
__device__ __forceinline__ double wave_scan(double x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double y = __shfl_up(x, m, 64);
    if (lane >= m) x += y;
  }
  return x;
}
__device__ __forceinline__ float exp2_of(double x) { return __builtin_amdgcn_exp2f((float)x); }

// acc += A B over the plane pairs that count.
template <int NA, int NB>
__device__ __forceinline__ void mma(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], floatx4& acc) {
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      if (i + j < 3) acc = mfma16(a[i], b[j], acc);
}

// How the sequences of a launch are cut into segments of whole chunks, one workgroup
// (and block of z rows) each, and where the segments' states are.
struct Span {
  int segs, chunks;      // segments of a chain, chunks of a segment (the last one: fewer)
  int writes;            // segments, in walking order, whose own write is formed
  float* states;         // [chain][writes + 1][state]: the write of segment j in slot
                         // j + 1, then the state that segment j starts from in slot j
  float* decays;         // [chain][writes]: a segment's whole decay
};
// units: workgroups of one segment over all chains; most: chunks of a segment at most.
// Segments until some 768 workgroups run, of four chunks at least.
inline Span cut(long units, long seqlen, long most) {
  const long chunks = (seqlen + C - 1) / C;
  long n = units < 768 ? 768 / units : 1;
  if (n > chunks / 4) n = chunks / 4 > 1 ? chunks / 4 : 1;
  long per = (chunks + n - 1) / n;
  if (per > most) per = most;
  return Span{(int)((chunks + per - 1) / per), (int)per, 0, nullptr, nullptr};
}

// Workgroup x of a launch: value-row block and unit (chain, segment), the row blocks of
// one unit 8 apart, so that they share the q and k rows in one XCD's L2.
__device__ __forceinline__ bool place(int blocks, long units, int& block, long& unit) {
  const long x = blockIdx.x;
  block = (int)((x / 8) % blocks);
  unit = (x / 8 / blocks) * 8 + x % 8;
  return unit < units;
}
inline unsigned grid_of(int blocks, long units) { return (unsigned)((units + 7) / 8 * 8 * blocks); }

// z rows of a workgroup: 64, or 32 where both x and z are float32 and the planes at 128
// columns would not fit the LDS.
template <typename TX, typename TZ, int DX>
constexpr int most_rows() { return sizeof(TX) == 4 && sizeof(TZ) == 4 && DX == 128 ? 32 : 64; }
inline int rows_of(bool both_f32, int dx, int nz) {
  const int most = both_f32 && dx == 128 ? 32 : 64;
  return nz < most ? nz : most;
}

}  // namespace gated
}  // namespace falcon
