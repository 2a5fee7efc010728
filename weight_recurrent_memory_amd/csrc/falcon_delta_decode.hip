// falcon_delta_decode.hip - one decode step of the gated delta rule.
//
// Per (sequence, head), a = exp(log_a), b = beta:
//   u = b (v - a S k),   S' = a S + u k^T   (in place),   o = S' q = a (S q) + u (k . q)
// Every row of S (a value channel) is updated and read by itself, so one pass reads S,
// forms S k and S q, writes S' and o, and a head's rows may be split over workgroups.
// Bound by HBM: 8 dk dv bytes of state per head, under one flop per byte.  A row lies on
// dk / 4 lanes, 16 bytes each.  512 x 12 x 64 x 64: 34.9 us a step = 5.9 TB/s (part of the 100 MB state
// stays in the Infinity Cache between steps; a copy of 1 GiB moves 5.1 to 5.25 TB/s);
// 1 x 12 x 128 x 128: 3.0 us, a launch's latency (9.3 us a call with the binding's host time).
#include "falcon_block_launch.h"
#include "falcon_gated.h"

namespace falcon {
namespace {

// 16 rows a workgroup: 4 dk threads, one launch shape for few heads (whose rows then lie
// on many compute units) and for many.
constexpr int kRows = 16;

template <typename T, int DK>
__global__ __launch_bounds__(kRows * DK / 4) void delta_decode_kernel(DeltaDecodeArgs a) {
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
  const float vv = ld_in(v, head * a.dv + row), b = a.beta[head];
  // (what counts as a reset is the sequence form's rule)
  const float la = a.log_a ? a.log_a[head] : 0.0f, dec = gated::is_reset(la) ? 0.0f : expf(la);
  const float sk = group_sum<TPR>(s.x * kk[0] + s.y * kk[1] + s.z * kk[2] + s.w * kk[3]);
  const float u = b * (vv - dec * sk);
  floatx4 n;
  n.x = dec * s.x + u * kk[0];
  n.y = dec * s.y + u * kk[1];
  n.z = dec * s.z + u * kk[2];
  n.w = dec * s.w + u * kk[3];
  __builtin_nontemporal_store(n, reinterpret_cast<floatx4*>(Sh));
  const float kq = group_sum<TPR>(kk[0] * qq[0] + kk[1] * qq[1] + kk[2] * qq[2] + kk[3] * qq[3]);
  const float sq = group_sum<TPR>(s.x * qq[0] + s.y * qq[1] + s.z * qq[2] + s.w * qq[3]);
  if (threadIdx.x % TPR == 0) a.o[head * a.dv + row] = dec * sq + u * kq;
}

template <typename T, int DK>
hipError_t go(const DeltaDecodeArgs& a, hipStream_t stream) {
  const long blocks = (long)a.nseq * a.heads * (a.dv / kRows);
  hipLaunchKernelGGL((delta_decode_kernel<T, DK>), dim3((unsigned)blocks), dim3(kRows * DK / 4), 0, stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t with_dk(const DeltaDecodeArgs& a, hipStream_t stream) {
  switch (a.dk) {
    case 16: return go<T, 16>(a, stream);
    case 32: return go<T, 32>(a, stream);
    case 64: return go<T, 64>(a, stream);
    case 128: return go<T, 128>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_delta_decode(const DeltaDecodeArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  return a.dtype == 0 ? with_dk<uint16_t>(a, stream) : with_dk<float>(a, stream);
}

}  // namespace falcon
