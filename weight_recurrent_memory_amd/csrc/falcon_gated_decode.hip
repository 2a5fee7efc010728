// falcon_gated_decode.hip - one decode step of the gated linear recurrence.
//
// Per (sequence, head), a = exp(log_a):
//   S' = a S + v k^T   (in place),   o = S' q = a (S q) + v (k . q)
// Every row of S (a value channel) is updated and read by itself, so one pass
// reads S, writes S' and forms o, and a head's rows may be split over
// workgroups.  Bound by HBM: 8 dk dv bytes of state per head, ~1/2 flop per
// byte.  A row lies on dk / 4 lanes, 16 bytes each; all loads of a lane are
// issued before the first sum.
#include "falcon_device.h"
#include "falcon_launch.h"

namespace falcon {
namespace {

// Rows of a workgroup of NT threads: NT / (dk / 4) in a pass.
template <typename T, int DK, int NT, int PASSES>
__global__ __launch_bounds__(NT) void gated_decode_kernel(GatedDecodeArgs a) {
  constexpr int TPR = DK / 4, RPP = NT / TPR, ROWS = RPP * PASSES;
  const T* __restrict__ q = static_cast<const T*>(a.q);
  const T* __restrict__ k = static_cast<const T*>(a.k);
  const T* __restrict__ v = static_cast<const T*>(a.v);
  const int blocks = a.dv / ROWS;                       // row blocks of a head
  const long head = blockIdx.x / blocks;
  const int row0 = (int)(blockIdx.x % blocks) * ROWS + (int)threadIdx.x / TPR;
  const int c0 = (threadIdx.x % TPR) * 4;
  float* __restrict__ Sh = a.S + (head * a.dv + row0) * DK + c0;

  floatx4 s[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p)
    s[p] = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(Sh + p * RPP * DK));
  float kk[4], qq[4], vv[PASSES];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    kk[e] = ld_in(k, head * DK + c0 + e);
    qq[e] = ld_in(q, head * DK + c0 + e);
  }
#pragma unroll
  for (int p = 0; p < PASSES; ++p) vv[p] = ld_in(v, head * a.dv + row0 + p * RPP);
  const float dec = a.log_a ? expf(a.log_a[head]) : 1.0f;
  const float kq = group_sum<TPR>(kk[0] * qq[0] + kk[1] * qq[1] + kk[2] * qq[2] + kk[3] * qq[3]);
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const float sq =
        group_sum<TPR>(s[p].x * qq[0] + s[p].y * qq[1] + s[p].z * qq[2] + s[p].w * qq[3]);
    floatx4 n;
    n.x = dec * s[p].x + vv[p] * kk[0];
    n.y = dec * s[p].y + vv[p] * kk[1];
    n.z = dec * s[p].z + vv[p] * kk[2];
    n.w = dec * s[p].w + vv[p] * kk[3];
    __builtin_nontemporal_store(n, reinterpret_cast<floatx4*>(Sh + p * RPP * DK));
    if (threadIdx.x % TPR == 0) a.o[head * a.dv + row0 + p * RPP] = dec * sq + vv[p] * kq;
  }
}

template <typename T, int DK, int NT, int PASSES>
hipError_t go(const GatedDecodeArgs& a, hipStream_t stream) {
  const long blocks = (long)a.nseq * a.heads * (a.dv / (NT / (DK / 4) * PASSES));
  hipLaunchKernelGGL((gated_decode_kernel<T, DK, NT, PASSES>), dim3((unsigned)blocks), dim3(NT), 0,
                     stream, a);
  return hipGetLastError();
}

// 16 rows a workgroup: 16 * dk / 4 threads (64 at dk = 16, 512 at dk = 128).
template <typename T>
hipError_t with_dk(const GatedDecodeArgs& a, hipStream_t stream) {
  switch (a.dk) {
    case 16: return go<T, 16, 64, 1>(a, stream);
    case 32: return go<T, 32, 128, 1>(a, stream);
    case 64: return go<T, 64, 256, 1>(a, stream);
    case 128: return go<T, 128, 512, 1>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_gated_decode(const GatedDecodeArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  return a.dtype == 0 ? with_dk<uint16_t>(a, stream) : with_dk<float>(a, stream);
}

}  // namespace falcon
