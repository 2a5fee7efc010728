// falcon_rotary.hip - rotary positions at a block's entry: the norm of falcon_norm.hip's
// norm_in with the first rot columns of q and k turned in pairs by position * frequency.
//
//   rotary_in      x = q_in / sqrt(|q_in|^2 + eps);  a pair (x1, x2) of columns becomes
//                  scale (x1 cos - x2 sin, x2 cos + x1 sin);  k likewise;  v = v_in
//   rotary_in_bwd  dy turned by the opposite angle and scaled, then
//                  dx = r (dy - y (y . dy)),  y = r x,  r = 1 / sqrt(|x|^2 + eps)
//
// Bound by HBM like the norms.  A position times a frequency passes 2^24 radians in a long
// document and keeps no fraction in float32: angles are formed in two float64, as turns, and
// reduced there (in one, an angle at 2^53 is off by a radian); the fraction of a turn then goes to
// sincospi in float32.  A workgroup
// forms them once per token of its tile, in LDS, for all heads; its first rows are on their way
// meanwhile.  Measured: 8x2048x12x64 bf16 33 us = 4.6 TB/s (norm_in, without the rotation, 26 us),
// 1x8191x8x128 float32 37 us = 5.4 TB/s over the outputs of the call before, which the Infinity Cache
// still holds (rows not read ahead: 40), and 46 us into other memory; the gradient at
// 4x1999x16x128 bf16 64 us = 5.7 TB/s (norm_in_bwd 60), 512 single tokens x 12 x 64 5.2 us.
#include "falcon_block_launch.h"
#include "falcon_rows.h"

namespace falcon {
using namespace rows;
namespace {

// 16 bytes of a row on their way, 0 where there is no row, and their values.
template <typename T>
__device__ __forceinline__ uint4 fetch(const T* x, bool in, long at) {
  return in ? *reinterpret_cast<const uint4*>(x + at) : uint4{0u, 0u, 0u, 0u};
}
template <typename T>
__device__ __forceinline__ void floats_of(const uint4& u, float (&x)[Vec<T>::V]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}

template <int D, int TT>
struct Angles {
  alignas(16) float cos[TT][D / 2];
  alignas(16) float sin[TT][D / 2];
};

// position * freq as a fraction of a turn, at most 1/2: products as a value and what rounding took
// from it, 1 / (2 pi) to 106 bits, so good to 2^-52 of a turn up to 2^53 turns.
__device__ __forceinline__ double turns_of(double position, double freq) {
#pragma clang fp contract(off)
  const double c = 0.15915494309189535, c_rest = -9.839338337591243e-18;
  const double a = position * freq, a_rest = __builtin_fma(position, freq, -a);
  const double t = a * c, t_rest = __builtin_fma(a, c, -t) + __builtin_fma(a, c_rest, a_rest * c);
  const double x = (t - rint(t)) + t_rest;
  return x - rint(x);
}

// cos and sin, scaled, of the tile's tokens and the rotation's pairs.
template <int D, int TT>
__device__ __forceinline__ void angles_of(Angles<D, TT>& a, const Rotation& r, long tile, long N) {
  const int h = r.rot / 2;
  for (int i = threadIdx.x; i < TT * h; i += NT) {
    const int t = i / h, p = i % h;
    const long n = tile * TT + t;
    float s = 0.0f, c = 1.0f;
    if (n < N) {
      sincospif((float)(2.0 * turns_of((double)r.positions[n], r.freqs[p])), &s, &c);
    }
    a.cos[t][p] = r.scale * c;
    a.sin[t][p] = r.scale * s;
  }
}

// The turned columns of V at column c of a row; sign -1 turns back.  `row`: the wave's
// scratch of 64 V floats.
template <int V, int VPR>
__device__ __forceinline__ void turn(float (&x)[V], int c, const float* cs, const float* sn, int rot, int pairs,
                                     float sign, float* row) {
  if (pairs == 1) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      if (c + i < rot) {
        const float co = cs[(c + i) / 2], si = sign * sn[(c + i) / 2];
        const float a = x[i], b = x[i + 1];
        x[i] = a * co - b * si;
        x[i + 1] = b * co + a * si;
      }
    }
    return;
  }
  const int h = rot / 2;
  float y[V];
  if (h % V == 0) {
    // a lane's partners lie together on another lane of the row
    const int lane = threadIdx.x & 63;
    const int from = c >= rot ? lane : c < h ? lane + h / V : lane - h / V;
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = __shfl(x[i], from, 64);
  } else {
    const int lane = threadIdx.x & 63, first = (lane / VPR) * VPR * V;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < V; ++i) row[lane * V + i] = x[i];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = c + i;
      y[i] = row[first + (j >= rot ? j : j < h ? j + h : j - h)];
    }
    __builtin_amdgcn_wave_barrier();
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = c + i;
    if (j < rot) {
      const int p = j < h ? j : j - h;
      const float si = sign * sn[p];
      x[i] = x[i] * cs[p] + (j < h ? -y[i] : y[i]) * si;
    }
  }
}

template <typename T, int D, int TT>
struct RotaryLds {
  Angles<D, TT> a;
  float row[NT / 64][64 * Vec<T>::V];
};

// Rows of q or k (TURN), or v's copied.
template <typename T, int D, int TT, bool TURN>
__device__ __forceinline__ void rotary_in_rows(const T* x, long ld, T* y, const RotaryInArgs& a, void* smem) {
  constexpr int V = Vec<T>::V, VPR = D / V, RPP = NT / VPR;
  RotaryLds<T, D, TT>& lds = *static_cast<RotaryLds<T, D, TT>*>(smem);
  const int c = (threadIdx.x % VPR) * V;
  const long N = (long)a.batch * a.seqlen;
  const int rows = TT * a.heads;
  for (long tile = blockIdx.x; tile * TT < N; tile += gridDim.x) {
    Row next = row_at<TT>(tile, (int)threadIdx.x / VPR, N, a.heads, a.seqlen);
    uint4 raw = fetch<T>(x, next.in, next.tok * ld + (long)next.h * D + c);
    if (TURN) {
      __syncthreads();
      angles_of<D, TT>(lds.a, a.r, tile, N);
      __syncthreads();
    }
    for (int r0 = 0; r0 < rows; r0 += RPP) {
      const int at = r0 + (int)threadIdx.x / VPR;
      const Row w = next;
      float f[V];
      floats_of<T>(raw, f);
      if (r0 + RPP < rows) {
        next = row_at<TT>(tile, at + RPP, N, a.heads, a.seqlen);
        raw = fetch<T>(x, next.in, next.tok * ld + (long)next.h * D + c);
      }
      if (TURN) {
        if (a.r.normalize) {
          float s = 0.0f;
#pragma unroll
          for (int i = 0; i < V; ++i) s += f[i] * f[i];
          s = group_sum<VPR>(s);
          const float rs = rsqrtf(s + a.eps);
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] *= rs;
        }
        turn<V, VPR>(f, c, lds.a.cos[at % TT], lds.a.sin[at % TT], a.r.rot, a.r.pairs, 1.0f,
                     lds.row[threadIdx.x >> 6]);
      }
      if (w.in) Vec<T>::store(y + w.head * D + c, f);
    }
  }
}

template <typename T, int DK, int DV, int TT>
__global__ __launch_bounds__(NT) void rotary_in_kernel(RotaryInArgs a) {
  __shared__ __align__(16) unsigned char smem[sizeof(RotaryLds<T, DK, TT>)];
  if (blockIdx.y == 0)
    rotary_in_rows<T, DK, TT, true>(static_cast<const T*>(a.q_in), a.ld_q, static_cast<T*>(a.q), a, smem);
  else if (blockIdx.y == 1)
    rotary_in_rows<T, DK, TT, true>(static_cast<const T*>(a.k_in), a.ld_k, static_cast<T*>(a.k), a, smem);
  else
    rotary_in_rows<T, DV, TT, false>(static_cast<const T*>(a.v_in), a.ld_v, static_cast<T*>(a.v), a, smem);
}

template <typename T, int D, int TT, bool TURN>
__device__ __forceinline__ void rotary_in_bwd_rows(const T* x, long ldx, const float* dy, T* dx, long ld,
                                                   const RotaryInBwdArgs& a, void* smem) {
  constexpr int V = Vec<T>::V, VPR = D / V, RPP = NT / VPR;
  RotaryLds<T, D, TT>& lds = *static_cast<RotaryLds<T, D, TT>*>(smem);
  const int c = (threadIdx.x % VPR) * V;
  const long N = (long)a.batch * a.seqlen;
  const int rows = TT * a.heads;
  for (long tile = blockIdx.x; tile * TT < N; tile += gridDim.x) {
    if (TURN) {
      __syncthreads();
      angles_of<D, TT>(lds.a, a.r, tile, N);
      __syncthreads();
    }
    for (int r0 = 0; r0 < rows; r0 += RPP) {
      const int at = r0 + (int)threadIdx.x / VPR;
      const Row w = row_at<TT>(tile, at, N, a.heads, a.seqlen);
      float f[V], g[V];
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = g[i] = 0.0f;
      if (w.in) {
        load_once<V>(dy + w.head * D + c, g);
        if (TURN && a.r.normalize) Vec<T>::load(x + w.tok * ldx + (long)w.h * D + c, f);
      }
      if (TURN) {
        turn<V, VPR>(g, c, lds.a.cos[at % TT], lds.a.sin[at % TT], a.r.rot, a.r.pairs, -1.0f,
                     lds.row[threadIdx.x >> 6]);
        if (a.r.normalize) {
          float s = 0.0f;
#pragma unroll
          for (int i = 0; i < V; ++i) s += f[i] * f[i];
          s = group_sum<VPR>(s);
          const float rs = rsqrtf(s + a.eps);
          float dot = 0.0f;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            f[i] *= rs;
            dot += f[i] * g[i];
          }
          dot = group_sum<VPR>(dot);
#pragma unroll
          for (int i = 0; i < V; ++i) g[i] = rs * (g[i] - f[i] * dot);
        }
      }
      if (w.in) store_once<T, V>(dx + w.tok * ld + (long)w.h * D + c, g);
    }
  }
}

template <typename T, int DK, int DV, int TT>
__global__ __launch_bounds__(NT) void rotary_in_bwd_kernel(RotaryInBwdArgs a) {
  __shared__ __align__(16) unsigned char smem[sizeof(RotaryLds<T, DK, TT>)];
  if (blockIdx.y == 0)
    rotary_in_bwd_rows<T, DK, TT, true>(static_cast<const T*>(a.q_in), a.ld_q, a.dq, static_cast<T*>(a.dq_in),
                                        a.ld_dq, a, smem);
  else if (blockIdx.y == 1)
    rotary_in_bwd_rows<T, DK, TT, true>(static_cast<const T*>(a.k_in), a.ld_k, a.dk, static_cast<T*>(a.dk_in),
                                        a.ld_dk, a, smem);
  else
    rotary_in_bwd_rows<T, DV, TT, false>(nullptr, 0, a.dv, static_cast<T*>(a.dv_in), a.ld_dv, a, smem);
}

// Tokens of a tile; calls of few tokens take 4, for more workgroups.
constexpr int kTile = 8, kTileFew = 4;
constexpr long kFewTokens = 4096;

// workgroups of a launch: one a tile, up to 2^20 (each then walks several tiles)
unsigned groups_of(long N) {
  const int tile = N < kFewTokens ? kTileFew : kTile;
  const long n = (N + tile - 1) / tile;
  return (unsigned)(n < (1l << 20) ? n : (1l << 20));
}

}  // namespace

hipError_t launch_rotary_in(const RotaryInArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  const long N = (long)a.batch * a.seqlen;
  const dim3 grid(groups_of(N), a.v ? 3 : 2);
  return with_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    return with_dim(a.dk, [&](auto dk) {
      return with_dim(a.dv, [&](auto dv) {
        if (N < kFewTokens)
          hipLaunchKernelGGL((rotary_in_kernel<T, dk(), dv(), kTileFew>), grid, dim3(NT), 0, stream, a);
        else
          hipLaunchKernelGGL((rotary_in_kernel<T, dk(), dv(), kTile>), grid, dim3(NT), 0, stream, a);
        return hipGetLastError();
      });
    });
  });
}

hipError_t launch_rotary_in_bwd(const RotaryInBwdArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  const long N = (long)a.batch * a.seqlen;
  const dim3 grid(groups_of(N), a.dv_in ? 3 : 2);
  return with_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    return with_dim(a.ndk, [&](auto dk) {
      return with_dim(a.ndv, [&](auto dv) {
        if (N < kFewTokens)
          hipLaunchKernelGGL((rotary_in_bwd_kernel<T, dk(), dv(), kTileFew>), grid, dim3(NT), 0, stream, a);
        else
          hipLaunchKernelGGL((rotary_in_bwd_kernel<T, dk(), dv(), kTile>), grid, dim3(NT), 0, stream, a);
        return hipGetLastError();
      });
    });
  });
}

}  // namespace falcon
