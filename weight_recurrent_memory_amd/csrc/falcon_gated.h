// falcon_gated.h - shared pieces of the gated recurrence's chunk kernels: operands as
// planes of bf16, their place in LDS, the sums of log decays.
//
// Planes.  An exact bf16 operand is one plane.  A float32 operand x is three: h =
// bf16(x), m = bf16(x - h), l = bf16(x - h - m), whose sum is x to 24 bits.  A product
// runs the plane pairs (i, j) with i + j < 3, so what is left out is 2^-24 of it: the
// matrix cores' bf16 rate (16 times the float32 one) at float32's precision, three
// passes with one float32 operand and six with two.
//
// Decays.  G_t = sum of log2 a over the chunk up to t, in float64 and kept as two floats:
// the decay from s to t is 2^(G_t - G_s), three additions and one v_exp.  In one float a
// reset (a log decay of -1000) would leave the differences behind it wrong by 2^-24 of
// 1000.  A decay is never divided by.
#pragma once
#include "falcon_device.h"
#include "falcon_launch.h"

namespace falcon {
namespace gated {

constexpr int C = 64;          // tokens of a chunk
constexpr int NT = 256;        // threads of a workgroup, 16 tokens of a chunk a wave

template <typename T>
constexpr int planes() { return sizeof(T) == 2 ? 1 : 3; }

// Element offset of (row, col) in a plane of rows of W (16 to 128) bf16: groups of 8
// elements (16 bytes) are XORed with bits of the row, so that the 16-byte reads of 8
// consecutive rows, of rows 0-3 and 8-11 together, and the transposed reads of 4 rows each
// fall into different banks.  Rows 16 apart are XORed alike: one address serves them all.
template <int W>
__device__ __forceinline__ int at(int row, int col) {
  const int f = (row & 7) ^ (((row >> 3) & 1) << 2);
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

// Place of row `row` among a chunk's 64 tokens (REV: the last token is row 0), and the
// token itself in the chunk of tokens t0..t0+63.
template <bool REV>
__device__ __forceinline__ int row_at(int row) { return REV ? C - 1 - row : row; }
template <bool REV>
__device__ __forceinline__ long token(long t0, int row) { return t0 + row_at<REV>(row); }

// The tokens of one chunk in one sequence, as a buffer: an offset behind the last token's
// row reads 0, whatever the row of the chunk.  Bases are the same for a whole wave, and
// the offsets inside a chunk are the same for every chunk.
typedef unsigned int uint4_t __attribute__((ext_vector_type(4)));
typedef unsigned int uint2_t __attribute__((ext_vector_type(2)));
struct Window {
  __amdgpu_buffer_rsrc_t r;
  // p: the first token's row; `rows` tokens are left in the sequence; rows `ld` elements
  // apart, of which the first `before` lie before p
  template <typename T>
  __device__ __forceinline__ Window(const T* p, long rows, int ld, int before) {
    const int n = (rows < C ? (int)rows : C) * ld - before;
    r = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), 0, n * (int)sizeof(T), 0x00027000);
  }
  __device__ __forceinline__ uint4 load16b(int at) const {
    const uint4_t u = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
    return uint4{u.x, u.y, u.z, u.w};
  }
  __device__ __forceinline__ uint2 load8b(int at) const {
    const uint2_t u = __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
    return uint2{u.x, u.y};
  }
  __device__ __forceinline__ unsigned load4b(int at) const {
    return __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
  }
};
constexpr int kNowhere = 1 << 30;      // an offset that reads 0

// Eight consecutive inputs as they are in memory, and as planes.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  uint4 u;
  __device__ __forceinline__ void load(const Window& w, int at) { u = w.load16b(at); }
  __device__ __forceinline__ void split(uint4 (&f)[1]) const { f[0] = u; }
};
template <>
struct Raw<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const Window& w, int at) {
    a = w.load16b(at);
    b = w.load16b(at + 16);
  }
  __device__ __forceinline__ void split(uint4 (&f)[3]) const {
    split3(__uint_as_float(a.x), __uint_as_float(a.y), f[0].x, f[1].x, f[2].x);
    split3(__uint_as_float(a.z), __uint_as_float(a.w), f[0].y, f[1].y, f[2].y);
    split3(__uint_as_float(b.x), __uint_as_float(b.y), f[0].z, f[1].z, f[2].z);
    split3(__uint_as_float(b.z), __uint_as_float(b.w), f[0].w, f[1].w, f[2].w);
  }
};
// Four consecutive inputs as they are in memory, and as floats.
template <typename T>
struct Raw4;
template <>
struct Raw4<uint16_t> {
  uint2 u;
  __device__ __forceinline__ void load(const Window& w, int at) { u = w.load8b(at); }
  __device__ __forceinline__ floatx4 values() const {
    return floatx4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                   __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u)};
  }
};
template <>
struct Raw4<float> {
  uint4 u;
  __device__ __forceinline__ void load(const Window& w, int at) { u = w.load16b(at); }
  __device__ __forceinline__ floatx4 values() const {
    return floatx4{__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
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


typedef short short4_t __attribute__((ext_vector_type(4)));

// One MFMA operand fragment (NP planes) of the transposed plane: columns col..col+15, one
// a lane of 16, and rows row..row+7 for each group of 16 lanes.  ds_read_b64_tr_b16: in a
// group of 16 lanes, lane i gives the address of 4 columns from 4 (i % 4) on of row i / 4,
// and lane i gets column i of the 4 rows.
template <int NP, int W>
__device__ __forceinline__ void frag_t(const uint16_t* p, int stride, int row, int col,
                                       bf16x8 (&f)[NP]) {
  typedef __attribute__((address_space(3))) short4_t* lds_ptr;
  const int m = threadIdx.x & 15;
  const int a = at<W>(row + (m >> 2), col + 4 * (m & 3)), b = at<W>(row + 4 + (m >> 2), col + 4 * (m & 3));
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    struct { short4_t lo, hi; } x;
    x.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + i * stride + a));
    x.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + i * stride + b));
    f[i] = __builtin_bit_cast(bf16x8, x);
  }
}

// A chunk's rows of one input on its way to LDS: units of 8 columns of a token.
template <typename T, int D, bool REV>
struct Stage {
  static constexpr int NP = planes<T>();
  static constexpr int G = D / 8, UNITS = C * G, N = (UNITS + NT - 1) / NT;
  Raw<T> r[N];
  int from[N];             // of the chunk's first token

  // rows of `ld` elements (REV: the last token is row 0)
  __device__ __forceinline__ explicit Stage(int ld) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = threadIdx.x + i * NT;
      from[i] = UNITS % NT == 0 || u < UNITS ? (row_at<REV>(u / G) * ld + 8 * (u % G)) * (int)sizeof(T) : kNowhere;
    }
  }
  __device__ __forceinline__ void load(const Window& w) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i].load(w, from[i]);
  }
  // to planes of rows W wide
  template <int W>
  __device__ __forceinline__ void store(uint16_t* rows) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = threadIdx.x + i * NT;
      if (UNITS % NT != 0 && u >= UNITS) continue;
      uint4 a[NP];
      r[i].split(a);
#pragma unroll
      for (int p = 0; p < NP; ++p)
        *reinterpret_cast<uint4*>(rows + p * C * W + at<W>(u / G, 8 * (u % G))) = a[p];
    }
  }
};

// One token's row (lane % 16 of the wave's 16) as a product's second operand.
template <typename T, int D, bool REV>
struct Row {
  static constexpr int NP = planes<T>(), N = (D + 31) / 32;
  Raw<T> r[N];
  int from;
  __device__ __forceinline__ Row() {
    const int lane = threadIdx.x & 63, col = 8 * (lane >> 4);
    from = D >= 32 || col < D ? (row_at<REV>(16 * (threadIdx.x >> 6) + (lane & 15)) * D + col) * (int)sizeof(T) : kNowhere;
  }
  __device__ __forceinline__ void load(const Window& w) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i].load(w, from + 32 * i * (int)sizeof(T));
  }
  __device__ __forceinline__ void frags(bf16x8 (&f)[N][NP]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint4 u[NP];
      r[i].split(u);
#pragma unroll
      for (int p = 0; p < NP; ++p) f[i][p] = __builtin_bit_cast(bf16x8, u[p]);
    }
  }
};

// log2 of a decay of log g: at least -1000 log2 e (and a NaN stays one).
__device__ __forceinline__ double log2_decay(float g) {
  g = g < -1000.0f ? -1000.0f : g;
  return (double)g * 1.4426950408889634;
}
// x of the lane that a DPP control names, 0 where it names none.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double x) {
  const long long u = __builtin_bit_cast(long long, x);
  const int lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, ((long long)hi << 32) | (unsigned int)lo);
}
// Inclusive sum over the lanes of a wave, first lane first: inside the rows of 16 lanes,
// then the rows' last lanes on to the rows behind.
__device__ __forceinline__ double wave_scan(double x) {
  x += dpp<0x111, 0xf>(x);      // row_shr 1, 2, 4, 8
  x += dpp<0x112, 0xf>(x);
  x += dpp<0x114, 0xf>(x);
  x += dpp<0x118, 0xf>(x);
  x += dpp<0x142, 0xa>(x);      // row_bcast 15 to rows 1 and 3
  x += dpp<0x143, 0xc>(x);      // row_bcast 31 to rows 2 and 3
  return x;
}
__device__ __forceinline__ float exp2_of(double x) { return __builtin_amdgcn_exp2f((float)x); }
// A token whose decay is 0: nothing passes from before it.
__device__ __forceinline__ bool is_reset(float g) { return exp2_of(log2_decay(g)) == 0.0f; }

// A sum of log2 decays as two floats, and the decay 2^(t - s): the difference of the first
// parts is exact where they are near each other and else good to 2^-24 of an exponent
// whose decay is small.
__device__ __forceinline__ float2 two_floats(double x) {
  const float h = (float)x;
  return float2{h, (float)(x - (double)h)};
}
__device__ __forceinline__ float decay(float2 t, float2 s) {
  return __builtin_amdgcn_exp2f((t.x - s.x) + (t.y - s.y));
}

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
// units: workgroups of one segment over all chains; slots: how many the GPU holds at once,
// which is what is aimed at; most: chunks of a segment at most; whole: sequences of fewer
// chunks are not cut (the extra launches would cost more).  Segments have two chunks at
// least.  Measured, us: 1x4x32771x128 forward 92 with 512 workgroups (what the GPU holds
// of that kernel) against 104 with 768; forward cut and whole, 1x8xLx64: L 512 20.5 and
// 15, L 768 21.5 and 21, L 1000 21.5 and 27, 8x12x512x64 27.5 and 20.5; two chunks against
// four: backward 1x5x4099x128x64 84 and 108.
inline Span cut(long units, long seqlen, long slots, long most, long whole) {
  const long chunks = (seqlen + C - 1) / C;
  long n = units < slots && chunks >= whole ? slots / units : 1;
  if (n > chunks / 2) n = chunks / 2 > 1 ? chunks / 2 : 1;
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

// z rows of a workgroup: 64, or less where chains and segments (of two chunks) alone leave
// compute units without work.  Each row block forms the scores anew, so a full GPU takes
// as few as it can.
inline int rows_of(int nz, long chains, long seqlen, long whole) {
  const long chunks = (seqlen + C - 1) / C, segs = chunks >= whole ? chunks / 2 : 1;
  int rows = nz < 64 ? nz : 64;
  while (rows > 16 && chains * segs * (nz / rows) < 256) rows /= 2;
  return rows;
}

}  // namespace gated
}  // namespace falcon
