// falcon_rows.h - rows of heads, token-major and head-major, as the norms and the rotary
// positions read and write them: one row (one token of one head, d elements) lies on d / V
// lanes, V elements each, and a workgroup takes tiles of TT consecutive tokens with every head.
#pragma once
#include <type_traits>

#include "falcon_device.h"

namespace falcon {
namespace rows {

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

}  // namespace rows
}  // namespace falcon
