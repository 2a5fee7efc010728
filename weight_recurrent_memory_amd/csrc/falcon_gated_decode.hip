// falcon_gated_decode.hip - one decode step of the gated linear recurrence.
//
// Per (sequence, head), a = exp(log_a):
//   S' = a S + v k^T   (in place),   o = S' q = a (S q) + v (k . q)
// Every row of S (a value channel) is updated and read by itself, so one pass
// reads S, writes S' and forms o, and a head's rows may be split over
// workgroups.  Bound by HBM: 8 dk dv bytes of state per head, ~1/2 flop per
// byte.  A row lies on dk / 4 lanes, 16 bytes each.  512 x 12 x 64 x 64: 34.4 us a step = 6.0 TB/s (part of the
// 100 MB state stays in the Infinity Cache between steps; a copy of 1 GiB moves 5.25 TB/s);
// 1 x 12 x 128 x 128: 2.9 us, a launch's latency.
#include "falcon_device.h"
#include "falcon_launch.h"

namespace falcon {
namespace {

// 16 rows a workgroup: 4 dk threads, one launch shape for few heads (whose rows then lie
// on many compute units) and for many.
constexpr int kRows = 16;

template <typename T, int DK>
__global__ __launch_bounds__(kRows * DK / 4) void gated_decode_kernel(GatedDecodeArgs a) {
  constexpr int TPR = DK / 4;
  const T* __restrict__ q = static_cast<const T*>(a.q);
  const T* __restrict__ k = static_cast<const T*>(a.k);
  const T* __restrict__ v = static_cast<const T*>(a.v);
  const int blocks = a.dv / kRows;                      // row blocks of a head
  const long head = blockIdx.x / blocks;
  const int row = (int)(blockIdx.x % blocks) * kRows + (int)threadIdx.x / TPR;
  const int c0 = (threadIdx.x % TPR) * 4;
  float* __restrict__ Sh = a.S + (head * a.dv + row) * DK + c0;

  const floatx4 s = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(Sh));
  float kk[4], qq[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    kk[e] = ld_in(k, head * DK + c0 + e);
    qq[e] = ld_in(q, head * DK + c0 + e);
  }
  const float vv = ld_in(v, head * a.dv + row);
  const float dec = a.log_a ? expf(a.log_a[head]) : 1.0f;
  const float kq = group_sum<TPR>(kk[0] * qq[0] + kk[1] * qq[1] + kk[2] * qq[2] + kk[3] * qq[3]);
  const float sq = group_sum<TPR>(s.x * qq[0] + s.y * qq[1] + s.z * qq[2] + s.w * qq[3]);
  floatx4 n;
  n.x = dec * s.x + vv * kk[0];
  n.y = dec * s.y + vv * kk[1];
  n.z = dec * s.z + vv * kk[2];
  n.w = dec * s.w + vv * kk[3];
  __builtin_nontemporal_store(n, reinterpret_cast<floatx4*>(Sh));
  if (threadIdx.x % TPR == 0) a.o[head * a.dv + row] = dec * sq + vv * kq;
}

template <typename T, int DK>
hipError_t go(const GatedDecodeArgs& a, hipStream_t stream) {
  const long blocks = (long)a.nseq * a.heads * (a.dv / kRows);
  hipLaunchKernelGGL((gated_decode_kernel<T, DK>), dim3((unsigned)blocks), dim3(kRows * DK / 4), 0, stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t with_dk(const GatedDecodeArgs& a, hipStream_t stream) {
  switch (a.dk) {
    case 16: return go<T, 16>(a, stream);
    case 32: return go<T, 32>(a, stream);
    case 64: return go<T, 64>(a, stream);
    case 128: return go<T, 128>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_gated_decode(const GatedDecodeArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  return a.dtype == 0 ? with_dk<uint16_t>(a, stream) : with_dk<float>(a, stream);
}

}  // namespace falcon
