// falcon_block_launch.h - internal interface between the C layer of libfalcon_block
// (falcon_block_api.cpp) and the kernel launchers.  Arguments are already validated.
#pragma once
#include <hip/hip_runtime.h>

namespace falcon {

// ---- the gated delta rule over a sequence
struct DeltaArgs {
  int batch, heads, seqlen, dk, dv;
  int dtype;               // 0 bf16, 1 fp32
  const void* q;
  const void* k;
  const void* v;
  const float* beta;
  const float* log_a;      // may be null
  const float* S0;         // may be null
  float* o;
  float* S_out;            // may be null
  void* workspace;         // delta_workspace_bytes(...)
};
// (sizes and type count)
size_t delta_workspace_bytes(const DeltaArgs& a);
// Whether every launch has fewer than 2^32 work-items, the most that HIP takes.
bool delta_fits(const DeltaArgs& a);
hipError_t launch_delta(const DeltaArgs& a, hipStream_t stream);
struct DeltaBwdArgs {
  int batch, heads, seqlen, ndk, ndv;
  int dtype;
  const void* q;
  const void* k;
  const void* v;
  const float* beta;
  const float* log_a;      // may be null
  const float* S0;         // may be null
  const float* dO;
  const float* dS_L;       // may be null
  float* dq;
  float* dk;
  float* dv;
  float* dbeta;
  float* dlog_a;           // may be null; null where log_a is
  float* dS0;              // may be null
  void* workspace;         // delta_bwd_workspace_bytes(...)
};
size_t delta_bwd_workspace_bytes(const DeltaBwdArgs& a);
bool delta_bwd_fits(const DeltaBwdArgs& a);
hipError_t launch_delta_bwd(const DeltaBwdArgs& a, hipStream_t stream);
struct DeltaDecodeArgs {
  int nseq, heads, dk, dv;
  int dtype;
  float* S;
  const void* q;
  const void* k;
  const void* v;
  const float* beta;
  const float* log_a;      // may be null
  float* o;
};
hipError_t launch_delta_decode(const DeltaDecodeArgs& a, hipStream_t stream);

// ---- rotary positions at a block's entry; ld_*: elements from one token's row of heads to
// the next
struct Rotation {
  const long long* positions;   // [batch, L]
  const double* freqs;          // [rot / 2], radians a token
  int rot, pairs;               // pairs: 0 halves, 1 neighbours
  float scale;
  int normalize;
};
struct RotaryInArgs {
  int batch, heads, seqlen, dk, dv;
  int dtype;
  Rotation r;
  float eps;
  const void* q_in;
  long ld_q;
  const void* k_in;
  long ld_k;
  const void* v_in;        // null with v
  long ld_v;
  void* q;
  void* k;
  void* v;
};
struct RotaryInBwdArgs {
  int batch, heads, seqlen, ndk, ndv;
  int dtype;
  Rotation r;
  float eps;
  const void* q_in;
  long ld_q;
  const void* k_in;
  long ld_k;
  const float* dq;
  const float* dk;
  const float* dv;         // null with dv_in
  void* dq_in;
  long ld_dq;
  void* dk_in;
  long ld_dk;
  void* dv_in;
  long ld_dv;
};
hipError_t launch_rotary_in(const RotaryInArgs& a, hipStream_t stream);
hipError_t launch_rotary_in_bwd(const RotaryInBwdArgs& a, hipStream_t stream);

}  // namespace falcon
