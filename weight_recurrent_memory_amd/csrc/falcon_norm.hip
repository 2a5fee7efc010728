// falcon_norm.hip - the norms before and after a fast-weight block.
//
//   norm_in      q = q_in / sqrt(|q_in|^2 + eps), k likewise, v = v_in; from the
//                token-major rows of a projection to the head-major rows of the
//                sequence entry points
//   norm_in_bwd  with r = 1 / sqrt(|x|^2 + eps), y = r x:  dx = r (dy - y (y . dy))
//   norm_out     with r = 1 / sqrt(mean o^2 + eps), n = r o:
//                y = residual + scale act(gate) w n, head-major to token-major
//   norm_out_bwd with dz = scale dy act(gate):  dw = sum dz n,
//                dgate = scale dy w n act'(gate), dn = dz w,
//                dO = r (dn - n mean(n dn))
//
// All four are bound by HBM: a few operations per element, each element read
// and written once.  Measured (bf16), where a copy of 1 GiB moves 5.25 TB/s: norm_in
// 8x2048x12x64 26.1 us = 5.8 TB/s (the last call's rows are partly in the Infinity Cache),
// norm_in_bwd 4x1999x16x128 60.0 us = 6.0 TB/s, norm_out 8x2048x12x64 with gate and
// residual 26.0 us = 4.8 TB/s, norm_out_bwd 2x8192x16x128 100 us = 4.7 TB/s.
// One row (one token of one head, d elements) lies on d / V lanes, V elements each (one
// 16-byte access of the element type; float32 rows beside bf16 ones take two), so a
// row's sums are shuffles inside a lane group.  A workgroup takes a tile of TT consecutive tokens with every head and
// walks it head by head: the head-major side is then read or written in runs of
// TT rows, and the token-major side of a tile is one workgroup's, so that lines
// shared by two heads (d = 16: 32-byte rows) meet in one L2.
// Sums are float32; a result is rounded once, to the element type.
#include "falcon_device.h"
#include "falcon_launch.h"

#include <type_traits>

namespace falcon {
namespace {

constexpr int NT = 256;       // threads of a workgroup

// V consecutive elements of the element type as floats.
template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void load(const uint16_t* p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&x)[8]) {
    uint4 u;
    u.x = pack_bf16x2(x[0], x[1]);
    u.y = pack_bf16x2(x[2], x[3]);
    u.z = pack_bf16x2(x[4], x[5]);
    u.w = pack_bf16x2(x[6], x[7]);
    *reinterpret_cast<uint4*>(p) = u;
  }
};
template <>
struct Vec<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void load(const float* p, float (&x)[4]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = float4{x[0], x[1], x[2], x[3]};
  }
};

// The same stored past the caches, and V float32 values read past them, for
// norm_in_bwd, whose inputs have their last use there (4x1999x16x128: 60.8 us against 70.5;
// a block's forward and backward at 8x12x2048x64: 322 us against 328).  The other outputs
// are the next kernel's inputs: past the caches they cost it more than they save here.
template <typename T, int V>
__device__ __forceinline__ void store_once(T* p, const float (&x)[V]) {
  if constexpr (sizeof(T) == 4) {
    __builtin_nontemporal_store(floatx4{x[0], x[1], x[2], x[3]}, reinterpret_cast<floatx4*>(p));
  } else {
    typedef unsigned int uintx4 __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(uintx4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                       pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])},
                                reinterpret_cast<uintx4*>(p));
  }
}
template <int V>
__device__ __forceinline__ void load_once(const float* p, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const floatx4 u = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(p + i));
    x[i] = u.x; x[i + 1] = u.y; x[i + 2] = u.z; x[i + 3] = u.w;
  }
}

// V float32 values (16-byte aligned).
template <int V>
__device__ __forceinline__ void load_f32(const float* p, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 u = *reinterpret_cast<const float4*>(p + i);
    x[i] = u.x; x[i + 1] = u.y; x[i + 2] = u.z; x[i + 3] = u.w;
  }
}
template <int V>
__device__ __forceinline__ void store_f32(float* p, const float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4)
    *reinterpret_cast<float4*>(p + i) = float4{x[i], x[i + 1], x[i + 2], x[i + 3]};
}

// One row position of a tile: token n (flat over batch and length), head h.
struct Row {
  bool in;
  long tok;      // offset of the token-major row in units of ld, = n
  long head;     // head-major row index (b * H + h) * L + l
  int h;
};
template <int TT>
__device__ __forceinline__ Row row_at(long tile, int r, long N, int H, int L) {
  Row x;
  const int t = r % TT;
  x.h = r / TT;
  const long n = tile * TT + t;
  x.in = x.h < H && n < N;
  const uint32_t nn = x.in ? (uint32_t)n : 0u;    // N < 2^31
  const uint32_t b = nn / (uint32_t)L;
  x.tok = nn;
  x.head = ((long)b * H + (x.in ? x.h : 0)) * L + (nn - b * (uint32_t)L);
  return x;
}

// ---------------------------------------------------------------- norm_in

template <typename T, int D, int TT, bool NORM>
__device__ __forceinline__ void norm_in_rows(const T* x, long ld, T* y, const NormInArgs& a) {
  constexpr int V = Vec<T>::V, VPR = D / V, RPP = NT / VPR;
  const int c = (threadIdx.x % VPR) * V;
  const long N = (long)a.batch * a.seqlen;
  const int rows = TT * a.heads;
  for (long tile = blockIdx.x; tile * TT < N; tile += gridDim.x)
  for (int r0 = 0; r0 < rows; r0 += RPP) {
    const Row w = row_at<TT>(tile, r0 + (int)threadIdx.x / VPR, N, a.heads, a.seqlen);
    float f[V];
    if (w.in) {
      Vec<T>::load(x + w.tok * ld + (long)w.h * D + c, f);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = 0.0f;
    }
    if (NORM) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) s += f[i] * f[i];
      s = group_sum<VPR>(s);
      const float rs = rsqrtf(s + a.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] *= rs;
    }
    if (w.in) Vec<T>::store(y + w.head * D + c, f);
  }
}

template <typename T, int DK, int DV, int TT>
__global__ __launch_bounds__(NT) void norm_in_kernel(NormInArgs a) {
  if (blockIdx.y == 0)
    norm_in_rows<T, DK, TT, true>(static_cast<const T*>(a.q_in), a.ld_q, static_cast<T*>(a.q), a);
  else if (blockIdx.y == 1)
    norm_in_rows<T, DK, TT, true>(static_cast<const T*>(a.k_in), a.ld_k, static_cast<T*>(a.k), a);
  else
    norm_in_rows<T, DV, TT, false>(static_cast<const T*>(a.v_in), a.ld_v, static_cast<T*>(a.v), a);
}

template <typename T, int D, int TT, bool NORM>
__device__ __forceinline__ void norm_in_bwd_rows(const T* x, long ldx, const float* dy, T* dx,
                                                 long ld, const NormInBwdArgs& a) {
  constexpr int V = Vec<T>::V, VPR = D / V, RPP = NT / VPR;
  const int c = (threadIdx.x % VPR) * V;
  const long N = (long)a.batch * a.seqlen;
  const int rows = TT * a.heads;
  for (long tile = blockIdx.x; tile * TT < N; tile += gridDim.x)
  for (int r0 = 0; r0 < rows; r0 += RPP) {
    const Row w = row_at<TT>(tile, r0 + (int)threadIdx.x / VPR, N, a.heads, a.seqlen);
    float f[V], g[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = g[i] = 0.0f;
    if (w.in) {
      load_once<V>(dy + w.head * D + c, g);
      if (NORM) Vec<T>::load(x + w.tok * ldx + (long)w.h * D + c, f);
    }
    if (NORM) {
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
    if (w.in) store_once<T, V>(dx + w.tok * ld + (long)w.h * D + c, g);
  }
}

template <typename T, int DK, int DV, int TT>
__global__ __launch_bounds__(NT) void norm_in_bwd_kernel(NormInBwdArgs a) {
  if (blockIdx.y == 0)
    norm_in_bwd_rows<T, DK, TT, true>(static_cast<const T*>(a.q_in), a.ld_q, a.dq,
                                      static_cast<T*>(a.dq_in), a.ld_dq, a);
  else if (blockIdx.y == 1)
    norm_in_bwd_rows<T, DK, TT, true>(static_cast<const T*>(a.k_in), a.ld_k, a.dk,
                                      static_cast<T*>(a.dk_in), a.ld_dk, a);
  else
    norm_in_bwd_rows<T, DV, TT, false>(nullptr, 0, a.dv, static_cast<T*>(a.dv_in), a.ld_dv, a);
}

// --------------------------------------------------------------- norm_out

// s = 1 / (1 + e^-g) goes to 0 and 1 at the ends without a NaN
// (e^-g = inf gives 0; g s at g = -inf is kept out by the caller's finite gates).
__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

template <typename T, int D, int TT, bool GATE>
__global__ __launch_bounds__(NT) void norm_out_kernel(NormOutArgs a) {
  constexpr int V = Vec<T>::V, VPR = D / V, RPP = NT / VPR;
  const int c = (threadIdx.x % VPR) * V;
  const long N = (long)a.batch * a.seqlen;
  const int rows = TT * a.heads;
  const T* gate = static_cast<const T*>(a.gate);
  const T* res = static_cast<const T*>(a.residual);
  T* y = static_cast<T*>(a.y);
  float wv[V];
  load_f32<V>(a.weight + c, wv);
#pragma unroll
  for (int i = 0; i < V; ++i) wv[i] *= a.scale;
  for (long tile = blockIdx.x; tile * TT < N; tile += gridDim.x)
  for (int r0 = 0; r0 < rows; r0 += RPP) {
    const Row w = row_at<TT>(tile, r0 + (int)threadIdx.x / VPR, N, a.heads, a.seqlen);
    const long col = (long)w.h * D + c;
    float o[V], g[V], z[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = g[i] = z[i] = 0.0f;
    if (w.in) {
      load_f32<V>(a.o + w.head * D + c, o);
      if (GATE) Vec<T>::load(gate + w.tok * a.ld_gate + col, g);
      if (res) Vec<T>::load(res + w.tok * a.ld_res + col, z);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) s += o[i] * o[i];
    s = group_sum<VPR>(s);
    const float rs = rsqrtf(s * (1.0f / D) + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float t = o[i] * rs * wv[i];
      if (GATE) {
        const float sg = sigmoid(g[i]);
        t *= a.gate_kind == 0 ? g[i] * sg : sg;
      }
      z[i] += t;
    }
    if (w.in) Vec<T>::store(y + w.tok * a.ld_y + col, z);
  }
}

template <typename T, int D, int TT, bool GATE>
__global__ __launch_bounds__(NT) void norm_out_bwd_kernel(NormOutBwdArgs a, long tiles) {
  constexpr int V = Vec<T>::V, VPR = D / V, RPP = NT / VPR;
  __shared__ float part[RPP][D];
  const int c = (threadIdx.x % VPR) * V;
  const long N = (long)a.batch * a.seqlen;
  const int rows = TT * a.heads;
  const T* gate = static_cast<const T*>(a.gate);
  const T* dy = static_cast<const T*>(a.dy);
  T* dgate = static_cast<T*>(a.dgate);
  float wv[V], dw[V];
  load_f32<V>(a.weight + c, wv);
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = 0.0f;
  for (long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    for (int r0 = 0; r0 < rows; r0 += RPP) {
      const Row w = row_at<TT>(tile, r0 + (int)threadIdx.x / VPR, N, a.heads, a.seqlen);
      const long col = (long)w.h * D + c;
      float o[V], g[V], d[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = g[i] = d[i] = 0.0f;
      if (w.in) {
        load_f32<V>(a.o + w.head * D + c, o);
        if (GATE) Vec<T>::load(gate + w.tok * a.ld_gate + col, g);
        Vec<T>::load(dy + w.tok * a.ld_dy + col, d);
      }
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) s += o[i] * o[i];
      s = group_sum<VPR>(s);
      // (a lane group without a row adds 0 to dw also where eps = 0 makes its rsqrt infinite)
      const float rs = w.in ? rsqrtf(s * (1.0f / D) + a.eps) : 0.0f;
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        o[i] *= rs;                         // n
        d[i] *= a.scale;
        if (GATE) {
          const float e = expf(-g[i]), sg = 1.0f / (1.0f + e);
          // 1 - sg: as a difference it keeps ever fewer bits from g = 5 on and is 0 from 17 on
          const float rest = g[i] > 0.0f ? e * sg : 1.0f - sg;
          const float act = a.gate_kind == 0 ? g[i] * sg : sg;
          const float slope = a.gate_kind == 0 ? sg * (1.0f + g[i] * rest) : sg * rest;
          g[i] = d[i] * wv[i] * o[i] * slope;
          d[i] *= act;                      // dz
        }
        dw[i] += d[i] * o[i];
        d[i] *= wv[i];                      // dn
        dot += d[i] * o[i];
      }
      dot = group_sum<VPR>(dot) * (1.0f / D);
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = rs * (d[i] - o[i] * dot);
      if (w.in) {
        store_f32<V>(a.dO + w.head * D + c, o);
        if (GATE) Vec<T>::store(dgate + w.tok * a.ld_dgate + col, g);
      }
    }
  }
  // this workgroup's part of dw: its lane groups added in a fixed order
  const int grp = threadIdx.x / VPR;
#pragma unroll
  for (int i = 0; i < V; ++i) part[grp][c + i] = dw[i];
  __syncthreads();
  for (int j = threadIdx.x; j < D; j += NT) {
    float s = 0.0f;
    for (int g = 0; g < RPP; ++g) s += part[g][j];
    a.workspace[(long)blockIdx.x * D + j] = s;
  }
}

// dw = the sum of the workgroups' parts, in a fixed order: 16 columns a
// workgroup, 64 threads a column.
__global__ __launch_bounds__(1024) void norm_out_dweight_kernel(const float* part, int parts, int D,
                                                                float* dw) {
  __shared__ float sum[64][17];
  const int c = threadIdx.x % 16, g = threadIdx.x / 16;
  const int col = blockIdx.x * 16 + c;       // D is a multiple of 16
  float s = 0.0f;
#pragma unroll 8
  for (int p = g; p < parts; p += 64) s += part[(long)p * D + col];
  sum[g][c] = s;
  __syncthreads();
  for (int m = 32; m >= 1; m >>= 1) {
    if (g < m) sum[g][c] += sum[g + m][c];
    __syncthreads();
  }
  if (g == 0) dw[col] = sum[0][c];
}

// ---------------------------------------------------------------- launches

// Tokens of a tile.  norm_in with 8 against 16: 26.1 against 27.1 us (8x2048x12x64 bf16),
// its gradient 68 against 71 us (4x1999x16x128); norm_out with 16 against 8 and 32: 26.7
// against 26.8 and 28.5 us (8x2048x12x64 with gate and residual), its gradient with 8 and
// 2048 workgroups against 16 and 1024: 100 against 105 us (2x8192x16x128).  Calls of few
// tokens take 4, for more workgroups.
constexpr int kTileIn = 8, kTileOut = 16, kTileOutBwd = 8, kTileFew = 4;
constexpr long kFewTokens = 4096;
constexpr int kBwdGroups = 2048;  // workgroups of norm_out_bwd at most

int tile_of(long N, int tile) { return N < kFewTokens ? kTileFew : tile; }
long tiles_of(long N, int tile) { return (N + tile_of(N, tile) - 1) / tile_of(N, tile); }
// workgroups of a launch: one a tile, up to 2^20 (each then walks several tiles)
unsigned groups_of(long N, int tile) {
  const long n = tiles_of(N, tile);
  return (unsigned)(n < (1l << 20) ? n : (1l << 20));
}

// f(integral_constant<D>...) for a supported size
template <class F>
hipError_t with_dim(int d, F&& f) {
  switch (d) {
    case 16: return f(std::integral_constant<int, 16>());
    case 32: return f(std::integral_constant<int, 32>());
    case 64: return f(std::integral_constant<int, 64>());
    case 128: return f(std::integral_constant<int, 128>());
  }
  return hipErrorInvalidValue;
}
template <class F>
hipError_t with_type(int dtype, F&& f) {
  return dtype == 0 ? f(uint16_t()) : f(float());
}

}  // namespace

hipError_t launch_norm_in(const NormInArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  const long N = (long)a.batch * a.seqlen;
  const dim3 grid(groups_of(N, kTileIn), a.v ? 3 : 2);
  return with_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    return with_dim(a.dk, [&](auto dk) {
      return with_dim(a.dv, [&](auto dv) {
        if (tile_of(N, kTileIn) == kTileIn)
          hipLaunchKernelGGL((norm_in_kernel<T, dk(), dv(), kTileIn>), grid, dim3(NT), 0, stream, a);
        else
          hipLaunchKernelGGL((norm_in_kernel<T, dk(), dv(), kTileFew>), grid, dim3(NT), 0, stream, a);
        return hipGetLastError();
      });
    });
  });
}

hipError_t launch_norm_in_bwd(const NormInBwdArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  const long N = (long)a.batch * a.seqlen;
  const dim3 grid(groups_of(N, kTileIn), a.dv_in ? 3 : 2);
  return with_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    return with_dim(a.ndk, [&](auto dk) {
      return with_dim(a.ndv, [&](auto dv) {
        if (tile_of(N, kTileIn) == kTileIn)
          hipLaunchKernelGGL((norm_in_bwd_kernel<T, dk(), dv(), kTileIn>), grid, dim3(NT), 0, stream, a);
        else
          hipLaunchKernelGGL((norm_in_bwd_kernel<T, dk(), dv(), kTileFew>), grid, dim3(NT), 0, stream, a);
        return hipGetLastError();
      });
    });
  });
}

hipError_t launch_norm_out(const NormOutArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  const long N = (long)a.batch * a.seqlen;
  const dim3 grid(groups_of(N, kTileOut));
  return with_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    return with_dim(a.dv, [&](auto d) {
      auto go = [&](auto tile) {
        if (a.gate)
          hipLaunchKernelGGL((norm_out_kernel<T, d(), tile(), true>), grid, dim3(NT), 0, stream, a);
        else
          hipLaunchKernelGGL((norm_out_kernel<T, d(), tile(), false>), grid, dim3(NT), 0, stream, a);
        return hipGetLastError();
      };
      return tile_of(N, kTileOut) == kTileOut ? go(std::integral_constant<int, kTileOut>())
                                 : go(std::integral_constant<int, kTileFew>());
    });
  });
}

size_t norm_out_bwd_workspace_bytes(int batch, int seqlen, int dv) {
  const long tiles = tiles_of((long)batch * seqlen, kTileOutBwd);
  return (size_t)(tiles < kBwdGroups ? tiles : kBwdGroups) * dv * sizeof(float);
}

hipError_t launch_norm_out_bwd(const NormOutBwdArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  const long N = (long)a.batch * a.seqlen, tiles = tiles_of(N, kTileOutBwd);
  const int groups = (int)(tiles < kBwdGroups ? tiles : kBwdGroups);
  const hipError_t e = with_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    return with_dim(a.dv, [&](auto d) {
      auto go = [&](auto tile) {
        if (a.gate)
          hipLaunchKernelGGL((norm_out_bwd_kernel<T, d(), tile(), true>), dim3(groups), dim3(NT), 0, stream, a, tiles);
        else
          hipLaunchKernelGGL((norm_out_bwd_kernel<T, d(), tile(), false>), dim3(groups), dim3(NT), 0, stream, a, tiles);
        return hipGetLastError();
      };
      return tile_of(N, kTileOutBwd) == kTileOutBwd ? go(std::integral_constant<int, kTileOutBwd>())
                                 : go(std::integral_constant<int, kTileFew>());
    });
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_out_dweight_kernel, dim3(a.dv / 16), dim3(1024), 0, stream, a.workspace,
                     groups, a.dv, a.dweight);
  return hipGetLastError();
}

}  // namespace falcon
