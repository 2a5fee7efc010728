// falcon_delta_solve.hip - T = (I + A)^-1 of every 64-token chunk of the gated delta rule,
// A_ts = b_t D_ts (k_t . k_s) for s < t.
//
// One wave a chunk, no barriers.  The scores k_s . k_t are matrix products; the four
// diagonal blocks of 16 are inverted by forward substitution, a column a lane (stable also
// where keys repeat and A's entries are 1, unlike a product of powers of A, whose entries
// grow to binomials); then blocks of 32 and of 64 from
//   [[X, 0], [C, Y]]^-1 = [[X^-1, 0], [-Y^-1 C X^-1, Y^-1]]
// on matrix cores, float32 operands as three bf16 planes.  T is written as the walk's
// operands (18 KB a chunk; the transposed ones for the gradients as much again).
// 8x12x2048x64 bf16: 21 us for the 32 chunks of each chain, 81 MB read and written = 3.9 TB/s (32 us with the
// transposed ones); one chunk alone takes 6.7 us.
#include "falcon_delta.h"

namespace falcon {
namespace delta {
namespace {

constexpr int kPitch = 68;          // floats of a row of T in LDS: 16-byte reads of 16 rows fall apart
constexpr int kDiag = 272;          // floats of a diagonal block: four blocks fall into different banks

struct SolveLds {
  alignas(16) float t[C * kPitch];  // first the diagonal blocks of A, then T
  alignas(16) float2 g[C];
  alignas(16) float b[C];
};

__device__ __forceinline__ constexpr int tri(int i, int j) { return i * (i + 1) / 2 + j; }

// Rows row0 + m of T, columns in paired order from col0 on (pairs: also col0 + 16 ..).
__device__ __forceinline__ void rows_of_T(const float* t, int row0, int col0, bool both, bf16x8 (&f)[3]) {
  const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  const float* p = t + (row0 + m) * kPitch + col0 + 4 * g;
  floatx4 hi = {0.f, 0.f, 0.f, 0.f};
  const floatx4 lo = *reinterpret_cast<const floatx4*>(p);
  if (both) hi = *reinterpret_cast<const floatx4*>(p + 16);
  frag_pair(lo, hi, f);
}
// Columns col0 + m, rows in paired order.
__device__ __forceinline__ void cols_of_T(const float* t, int row0, int col0, bool both, bf16x8 (&f)[3]) {
  const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  const float* p = t + (row0 + 4 * g) * kPitch + col0 + m;
  const floatx4 lo = {p[0], p[kPitch], p[2 * kPitch], p[3 * kPitch]};
  floatx4 hi = {0.f, 0.f, 0.f, 0.f};
  if (both) {
    p += 16 * kPitch;
    hi = floatx4{p[0], p[kPitch], p[2 * kPitch], p[3 * kPitch]};
  }
  frag_pair(lo, hi, f);
}

template <typename T, int DK>
__global__ __launch_bounds__(64 * kSolveWaves) void solve_kernel(SolveArgs a, int chunks) {
  constexpr int NP = planes<T>(), NQ = (DK + 31) / 32;
  __shared__ SolveLds all[kSolveWaves];
  SolveLds& lds = all[wave_id()];
  const long unit = (long)blockIdx.x * kSolveWaves + wave_id();
  if (unit >= a.chains * chunks) return;
  const long chain = unit / chunks, t0 = (unit % chunks) * C, len = a.seqlen;
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const floatx4 zero = {0.f, 0.f, 0.f, 0.f};

  GateLoad gl;
  gl.load(a.log_a ? a.log_a + chain * len : nullptr, a.beta + chain * len, t0, len);
  const T* k = static_cast<const T*>(a.k) + chain * len * DK;
  const Window wk(k + t0 * DK, len - t0, DK, 0);
  bf16x8 kf[4][NQ][NP];
  {
    PairRow<T, DK> row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i].load(wk, 16 * i + m);
    lds.g[lane] = two_floats(wave_scan(log2_decay(gl.raw)));
    lds.b[lane] = gl.beta;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int n = 0; n < NQ; ++n) row[i].frag(n, kf[i][n]);
  }
  wave_order();

  // A by tiles, transposed: rows s = 16 j + 4 g + r, columns t = 16 i + m
  floatx4 A[10];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 Gt = lds.g[16 * i + m];
    const float bt = lds.b[16 * i + m];
#pragma unroll
    for (int j = 0; j <= i; ++j) {
      floatx4 p = zero;
#pragma unroll
      for (int n = 0; n < NQ; ++n) mma<NP, NP>(kf[j][n], kf[i][n], p);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = bt * decay(Gt, lds.g[16 * j + 4 * g + r]) * p[r];
        A[tri(i, j)][r] = (j < i || 4 * g + r < m) ? x : 0.0f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<floatx4*>(lds.t + i * kDiag + m * 16 + 4 * g) = A[tri(i, i)];
  wave_order();
  // the diagonal blocks' inverses: lane = column m of block g
  float x[16];
  {
    const float* d = lds.t + g * kDiag;
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      float s0 = t == m ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
      for (int s4 = 0; s4 < t; s4 += 4) {
        const floatx4 row = *reinterpret_cast<const floatx4*>(d + t * 16 + s4);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (s4 + r < t) {
            if (r & 1) s1 -= row[r] * x[s4 + r];
            else s0 -= row[r] * x[s4 + r];
          }
      }
      x[t] = s0 + s1;
    }
  }
  wave_order();
  // (of the tiles above the diagonal two are read)
  *reinterpret_cast<floatx4*>(lds.t + m * kPitch + 16 + 4 * g) = zero;
  *reinterpret_cast<floatx4*>(lds.t + (32 + m) * kPitch + 48 + 4 * g) = zero;
#pragma unroll
  for (int t = 0; t < 16; ++t) lds.t[(16 * g + t) * kPitch + 16 * g + m] = x[t];
  wave_order();

  bf16x8 fa[3], fb[3];
  // blocks of 32
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 2 * h + 1, j = 2 * h;
    floatx4 y = zero, z = zero;
    frag_pair(A[tri(i, j)], zero, fa);
    cols_of_T(lds.t, 16 * j, 16 * j, false, fb);
    mma<3, 3>(fa, fb, y);
    frag_pair(y, zero, fb);
    rows_of_T(lds.t, 16 * i, 16 * i, false, fa);
    mma<3, 3>(fa, fb, z);
#pragma unroll
    for (int r = 0; r < 4; ++r) lds.t[(16 * i + 4 * g + r) * kPitch + 16 * j + m] = -z[r];
  }
  wave_order();
  // the block of 64's lower left
  floatx4 M[2][2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    cols_of_T(lds.t, 0, 16 * c, true, fb);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      frag_pair(A[tri(2 + i, 0)], A[tri(2 + i, 1)], fa);
      M[i][c] = zero;
      mma<3, 3>(fa, fb, M[i][c]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    rows_of_T(lds.t, 32 + 16 * i, 32, true, fa);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      floatx4 z = zero;
      frag_pair(M[0][c], M[1][c], fb);
      mma<3, 3>(fa, fb, z);
#pragma unroll
      for (int r = 0; r < 4; ++r) lds.t[(32 + 16 * i + 4 * g + r) * kPitch + 16 * c + m] = -z[r];
    }
  }
  wave_order();

  uint4* out = a.T + unit * kT + lane;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j <= i / 2; ++j) {
      rows_of_T(lds.t, 16 * i, 32 * j, true, fa);
#pragma unroll
      for (int p = 0; p < 3; ++p) out[(frag_of(i, j) * 3 + p) * 64] = __builtin_bit_cast(uint4, fa[p]);
    }
  if (!a.Tt) return;
  // of row tile 3 - i (a column of T) the 32-token steps 1 - j
  out = a.Tt + unit * kT + lane;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j <= i / 2; ++j) {
      cols_of_T(lds.t, 32 - 32 * j, 48 - 16 * i, true, fa);
#pragma unroll
      for (int p = 0; p < 3; ++p) out[(frag_of(i, j) * 3 + p) * 64] = __builtin_bit_cast(uint4, fa[p]);
    }
}

template <typename T>
hipError_t go(const SolveArgs& a, int dk, hipStream_t stream) {
  const int chunks = (int)(((long)a.seqlen + C - 1) / C);
  const long units = a.chains * chunks;
  return with_dim(dk, [&](auto d) {
    hipLaunchKernelGGL((solve_kernel<T, decltype(d)::value>), dim3((unsigned)((units + kSolveWaves - 1) / kSolveWaves)),
                       dim3(64 * kSolveWaves), 0, stream, a, chunks);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_solve(const SolveArgs& a, int dk, int dtype, hipStream_t stream) {
  return dtype == 0 ? go<uint16_t>(a, dk, stream) : go<float>(a, dk, stream);
}

}  // namespace delta
}  // namespace falcon
