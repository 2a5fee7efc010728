// falcon_launch.h - internal interface between the C-ABI layer (falcon_api.cpp)
// and the kernel launchers.  Arguments are already validated when these run.
#pragma once
#include <hip/hip_runtime.h>

namespace falcon {

// Arguments of one sequence call (recurrent or chunk form).
struct SeqArgs {
  int variant;       // falcon_variant
  int window;        // B
  int regression;    // 1: Falcon-1/2/3, 0: Falcon-1A/2A/3A
  float beta;        // scalar gain (beta_kind == 0)
  const void* beta_t;
  int beta_kind;     // 0 scalar, 1 per token, 2 per token and value channel
  float lambda, eps;
  int batch, heads, seqlen, dk, dv;
  int dtype;         // 0 bf16, 1 fp32
  const void* q;
  const void* k;
  const void* v;
  const void* k_prev;  // may be null
  const float* S0;     // may be null
  float* o;
  float* S_out;        // may be null
  int chunk;           // chunk form only
  // window history of a resumed Falcon-3/3A sequence: the window-1 samples
  // (x_j, y_j) before step 1, oldest first, [chain][window-1][dk or dv]; null:
  // none (zero samples)
  const void* x_hist = nullptr;
  const void* y_hist = nullptr;
  // sample pairing: x_t = k_{t - key_shift}; 1 = the previous key (x_1 = k_prev
  // or 0), 0 = the same step's key
  int key_shift = 1;
};

struct DecodeArgs {
  int regression;
  int window;        // 1, or B > 1 with x_hist / y_hist
  void* x_hist;      // [nseq*heads][window-1][dk], oldest first, updated in place
  void* y_hist;      // [nseq*heads][window-1][dv]
  float beta;
  const void* beta_t;
  int beta_kind;
  float lambda, eps;
  int nseq, heads, dk, dv;
  int dtype;
  float* S;
  void* k_prev;
  const void* q;
  const void* k;
  const void* v;
  float* o;
  int key_shift;     // 1: x = k_prev (then k_prev <- k); 0: x = k, k_prev unused
};

// Backward of the chunk form, windows 1..8 (falcon_backward.hip).
struct BwdArgs {
  int regression;
  int window;        // 1..8
  int key_shift;
  float beta;
  const void* beta_t;
  int beta_kind;
  float lambda, eps;
  int batch, heads;
  long seqlen;
  int ndk, ndv;      // sizes
  int dtype;
  const void* q;
  const void* k;
  const void* v;
  const void* k_prev;
  const float* S0;
  const float* dO;
  const float* dS_L;     // may be null
  const float* dk_last;  // may be null
  float* dq;
  float* dk;
  float* dv;
  float* dbeta_t;        // may be null
  float* dk_prev;        // may be null
  float* dS0;            // may be null
  float* workspace;      // backward_workspace_bytes(...)
};
size_t backward_workspace_bytes(int batch, int heads, long seqlen, int dk, int dv, int window);
// Largest per-chain buffer range the backward kernel addresses (bytes); the
// kernel needs it below 2^30.
size_t backward_chain_bytes(long seqlen, int dk, int dv, int window, int dtype);
hipError_t launch_backward(const BwdArgs& a, hipStream_t stream);

hipError_t launch_recurrent(const SeqArgs& a, hipStream_t stream);
// masked-parallel form, the whole call one masked system (falcon_masked.hip):
// seqlen 1..kMaskedMaxLen, window 1..8
constexpr int kMaskedMaxLen = 64;
hipError_t launch_masked(const SeqArgs& a, hipStream_t stream);
// workspace (optional): the two-kernel sliding-window form runs where it applies and
// ws_bytes >= chunk_wyb2_workspace_bytes(a)
hipError_t launch_chunk(const SeqArgs& a, hipStream_t stream, void* ws = nullptr, size_t ws_bytes = 0);
// window-1 chunk form, per-channel gains (falcon_chunk_w1.hip); cs = sub-chunk length
hipError_t launch_chunk_w1(const SeqArgs& a, hipStream_t stream, int cs);
// window-1 chunk form, gains shared by the value rows, dk in {32, 64}
// (falcon_chunk_wy.hip); 32-step chunks whatever the requested chunk
bool chunk_wy_supported(const SeqArgs& a);
hipError_t launch_chunk_wy(const SeqArgs& a, hipStream_t stream);
// sliding-window chunk form (window 2 or 4), gains shared by the value rows, dk in
// {64, 128} (falcon_chunk_wyb.hip); 16-step sub-chunks whatever the requested chunk
bool chunk_wyb_supported(const SeqArgs& a);
hipError_t launch_chunk_wyb(const SeqArgs& a, hipStream_t stream);
// the same in two kernels (regression family): a pre-pass writes every
// sub-chunk's folds to a workspace, a state kernel runs the sequential part;
// the workspace bytes it needs (0 where it does not apply) and its launch
size_t chunk_wyb2_workspace_bytes(const SeqArgs& a);
hipError_t launch_chunk_wyb2(const SeqArgs& a, void* workspace, hipStream_t stream);
// inner-product family, any window up to 16, gains shared by the value rows, dk in
// {64, 128}, dv a multiple of 32 (falcon_chunk_ip.hip); 64-step chunks
bool chunk_ip_supported(const SeqArgs& a);
hipError_t launch_chunk_ip(const SeqArgs& a, hipStream_t stream);
hipError_t launch_decode(const DecodeArgs& a, hipStream_t stream);
// the window-1 latest samples after a sequence call, written to x_out / y_out
// (which may equal a.x_hist / a.y_hist); enqueue after the call's kernel
hipError_t launch_history_out(const SeqArgs& a, void* x_out, void* y_out, hipStream_t stream);

// ---- gated linear recurrence (falcon_gated.hip, falcon_gated_bwd.hip)

// Forward over a sequence: S_t = a_t S_{t-1} + v_t k_t^T, o_t = S_t q_t, a = exp(log_a).
struct GatedArgs {
  int batch, heads, seqlen, dk, dv;
  int dtype;             // 0 bf16, 1 fp32
  const void* q;
  const void* k;
  const void* v;
  const float* log_a;    // may be null (no decay)
  const float* S0;       // may be null
  float* o;
  float* S_out;          // may be null
};
// Bytes of device workspace with which launch_gated cuts the sequence into segments
// (0: one segment in any case); without it every chain is one segment.
size_t gated_workspace_bytes(const GatedArgs& a);
hipError_t launch_gated(const GatedArgs& a, void* ws, size_t ws_bytes, hipStream_t stream);
struct GatedBwdArgs {
  int batch, heads, seqlen, ndk, ndv;
  int dtype;
  const void* q;
  const void* k;
  const void* v;
  const float* log_a;    // may be null
  const float* S0;       // may be null
  const float* dO;
  const float* dS_L;     // may be null
  float* dq;
  float* dk;
  float* dv;
  float* dlog_a;         // null exactly when log_a is
  float* dS0;            // may be null
  float* workspace;      // gated_bwd_workspace_bytes(...)
};
// (of the pointers only log_a, dS_L and dlog_a count, null or not)
size_t gated_bwd_workspace_bytes(const GatedBwdArgs& a);
hipError_t launch_gated_bwd(const GatedBwdArgs& a, hipStream_t stream);
struct GatedDecodeArgs {
  int nseq, heads, dk, dv;
  int dtype;
  float* S;
  const void* q;
  const void* k;
  const void* v;
  const float* log_a;    // may be null
  float* o;
};
hipError_t launch_gated_decode(const GatedDecodeArgs& a, hipStream_t stream);

// ---- norms before and after a block (falcon_norm.hip); ld_*: elements from one
// token's row of heads to the next

struct NormInArgs {
  int batch, heads, seqlen, dk, dv;
  int dtype;
  const void* q_in;
  long ld_q;
  const void* k_in;
  long ld_k;
  const void* v_in;      // null with v
  long ld_v;
  float eps;
  void* q;
  void* k;
  void* v;
};
struct NormInBwdArgs {
  int batch, heads, seqlen, ndk, ndv;
  int dtype;
  const void* q_in;
  long ld_q;
  const void* k_in;
  long ld_k;
  float eps;
  const float* dq;
  const float* dk;
  const float* dv;       // null with dv_in
  void* dq_in;
  long ld_dq;
  void* dk_in;
  long ld_dk;
  void* dv_in;
  long ld_dv;
};
struct NormOutArgs {
  int batch, heads, seqlen, dv;
  int dtype;
  const float* o;
  const float* weight;
  const void* gate;      // may be null
  long ld_gate;
  int gate_kind;         // 0 silu, 1 sigmoid
  const void* residual;  // may be null; may equal y
  long ld_res;
  float scale, eps;
  void* y;
  long ld_y;
};
struct NormOutBwdArgs {
  int batch, heads, seqlen, dv;
  int dtype;
  const float* o;
  const float* weight;
  const void* gate;      // null with dgate
  long ld_gate;
  int gate_kind;
  float scale, eps;
  const void* dy;
  long ld_dy;
  float* dO;
  void* dgate;
  long ld_dgate;
  float* dweight;
  float* workspace;      // norm_out_bwd_workspace_bytes(...)
};
hipError_t launch_norm_in(const NormInArgs& a, hipStream_t stream);
hipError_t launch_norm_in_bwd(const NormInBwdArgs& a, hipStream_t stream);
hipError_t launch_norm_out(const NormOutArgs& a, hipStream_t stream);
size_t norm_out_bwd_workspace_bytes(int batch, int seqlen, int dv);
hipError_t launch_norm_out_bwd(const NormOutBwdArgs& a, hipStream_t stream);

}  // namespace falcon
