// falcon_block_api.cpp - the C layer of libfalcon_block (declared in
// include/falcon_block.h): argument validation and launch on the caller's stream.
// Every check runs before the first HIP call.
#include "falcon_block.h"

#include "falcon_block_launch.h"
#include "falcon_check.h"

namespace {

// Records and workgroups are counted in 31 bits, a launch's work-items in 32.
bool delta_sizes(int batch, int heads, int seqlen, int dk, int dv) {
  return (double)batch * heads * (dk > dv ? dk : dv) * (((double)seqlen + 63.0) / 64.0) < 2147483648.0;
}
bool forward_sizes(int batch, int heads, int seqlen, int dk, int dv, int dtype) {
  return supported_dim(dk) && supported_dim(dv) && delta_sizes(batch, heads, seqlen, dk, dv) &&
         falcon::delta_fits(falcon::DeltaArgs{batch, heads, seqlen, dk, dv, dtype});
}
bool backward_sizes(int batch, int heads, int seqlen, int dk, int dv, int dtype) {
  return supported_dim(dk) && supported_dim(dv) && delta_sizes(batch, heads, seqlen, dk, dv) &&
         falcon::delta_bwd_fits(falcon::DeltaBwdArgs{batch, heads, seqlen, dk, dv, dtype});
}

}  // namespace

FALCON_EXPORT unsigned long long falcon_gated_delta_fwd_workspace_bytes(int batch, int heads, int seqlen,
                                                                        int dk, int dv, int dtype) {
  size_t N, es;
  if (check_sizes(batch, heads, seqlen, dk, dv, dtype, &N, &es) != FALCON_OK ||
      !forward_sizes(batch, heads, seqlen, dk, dv, dtype))
    return 0;
  falcon::DeltaArgs a{batch, heads, seqlen, dk, dv, dtype};
  return (unsigned long long)falcon::delta_workspace_bytes(a);
}

FALCON_EXPORT int falcon_gated_delta_fwd_chunk(int batch, int heads, int seqlen, int dk, int dv, int dtype,
                                               const void* q, const void* k, const void* v,
                                               const float* beta, const float* log_a, const float* S0,
                                               float* o, float* S_out, void* workspace,
                                               unsigned long long workspace_bytes, void* stream) {
  size_t N, es;
  int st = check_sizes(batch, heads, seqlen, dk, dv, dtype, &N, &es);
  if (st != FALCON_OK) return st;
  if (!q || !k || !v || !beta || !o || !workspace) return FALCON_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, S0, o, S_out, workspace};
  if (!all_aligned16(ptrs) || !aligned4(beta) || !aligned4(log_a)) return FALCON_ERR_INVALID_ARG;
  if (!forward_sizes(batch, heads, seqlen, dk, dv, dtype)) return FALCON_ERR_UNSUPPORTED;
  const falcon::DeltaArgs a{batch, heads, seqlen, dk, dv, dtype, q, k, v, beta, log_a, S0, o, S_out, workspace};
  const size_t need = falcon::delta_workspace_bytes(a);
  if (workspace_bytes < need) return FALCON_ERR_INVALID_ARG;
  const size_t NH = N * heads, state = (size_t)batch * heads * dv * dk * 4;
  const Range outs[] = {{o, NH * dv * 4}, {S_out, state}, {workspace, need}};
  const Range ins[] = {{q, NH * dk * es}, {k, NH * dk * es}, {v, NH * dv * es}, {beta, NH * 4}, {log_a, NH * 4}};
  if (any_overlap(outs, ins)) return FALCON_ERR_INVALID_ARG;
  const Range s0{S0, state};
  if (overlap(outs[0], s0) || overlap(outs[2], s0)) return FALCON_ERR_INVALID_ARG;
  if (S_out != S0 && overlap(outs[1], s0)) return FALCON_ERR_INVALID_ARG;
  return finish_launch(falcon::launch_delta(a, (hipStream_t)stream));
}

FALCON_EXPORT unsigned long long falcon_gated_delta_bwd_workspace_bytes(int batch, int heads, int seqlen,
                                                                        int dk, int dv, int dtype) {
  size_t N, es;
  if (check_sizes(batch, heads, seqlen, dk, dv, dtype, &N, &es) != FALCON_OK ||
      !backward_sizes(batch, heads, seqlen, dk, dv, dtype))
    return 0;
  falcon::DeltaBwdArgs a{batch, heads, seqlen, dk, dv, dtype};
  return (unsigned long long)falcon::delta_bwd_workspace_bytes(a);
}

FALCON_EXPORT int falcon_gated_delta_bwd_chunk(int batch, int heads, int seqlen, int dk, int dv, int dtype,
                                               const void* q, const void* k, const void* v,
                                               const float* beta, const float* log_a, const float* S0,
                                               const float* dO, const float* dS_L, float* dq, float* dk_out,
                                               float* dv_out, float* dbeta, float* dlog_a, float* dS0,
                                               void* workspace, unsigned long long workspace_bytes,
                                               void* stream) {
  size_t N, es;
  int st = check_sizes(batch, heads, seqlen, dk, dv, dtype, &N, &es);
  if (st != FALCON_OK) return st;
  if (!q || !k || !v || !beta || !dO || !dq || !dk_out || !dv_out || !dbeta || !workspace || (dlog_a && !log_a))
    return FALCON_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, S0, dO, dS_L, dq, dk_out, dv_out, dS0, workspace};
  if (!all_aligned16(ptrs) || !aligned4(beta) || !aligned4(log_a) || !aligned4(dbeta) || !aligned4(dlog_a))
    return FALCON_ERR_INVALID_ARG;
  if (!backward_sizes(batch, heads, seqlen, dk, dv, dtype)) return FALCON_ERR_UNSUPPORTED;
  const falcon::DeltaBwdArgs a{batch, heads, seqlen, dk, dv, dtype, q, k, v, beta, log_a, S0, dO, dS_L,
                               dq, dk_out, dv_out, dbeta, dlog_a, dS0, workspace};
  const size_t need = falcon::delta_bwd_workspace_bytes(a);
  if (workspace_bytes < need) return FALCON_ERR_INVALID_ARG;
  const size_t NH = N * heads, state = (size_t)batch * heads * dv * dk * 4;
  const Range outs[] = {{dq, NH * dk * 4}, {dk_out, NH * dk * 4}, {dv_out, NH * dv * 4}, {dbeta, NH * 4},
                        {dlog_a, NH * 4}, {dS0, state}, {workspace, need}};
  const Range ins[] = {{q, NH * dk * es}, {k, NH * dk * es}, {v, NH * dv * es}, {beta, NH * 4}, {log_a, NH * 4},
                       {S0, state}, {dO, NH * dv * 4}, {dS_L, state}};
  if (any_overlap(outs, ins)) return FALCON_ERR_INVALID_ARG;
  return finish_launch(falcon::launch_delta_bwd(a, (hipStream_t)stream));
}

FALCON_EXPORT int falcon_gated_delta_decode_step(int nseq, int heads, int dk, int dv, int dtype, float* S,
                                                 const void* q, const void* k, const void* v,
                                                 const float* beta, const float* log_a, float* o,
                                                 void* stream) {
  size_t N, es;
  int st = check_sizes(nseq, heads, 1, dk, dv, dtype, &N, &es);
  if (st != FALCON_OK) return st;
  if (!S || !q || !k || !v || !beta || !o) return FALCON_ERR_INVALID_ARG;
  const void* ptrs[] = {S, q, k, v, o};
  if (!all_aligned16(ptrs) || !aligned4(beta) || !aligned4(log_a)) return FALCON_ERR_INVALID_ARG;
  const size_t NH = N * heads;
  const Range outs[] = {{S, NH * dv * dk * 4}, {o, NH * dv * 4}};
  const Range ins[] = {{q, NH * dk * es}, {k, NH * dk * es}, {v, NH * dv * es}, {beta, NH * 4}, {log_a, NH * 4}};
  if (any_overlap(outs, ins)) return FALCON_ERR_INVALID_ARG;
  if (!supported_dim(dk) || !supported_dim(dv)) return FALCON_ERR_UNSUPPORTED;
  // one thread per four state elements in one launch
  if ((double)NH * dv * dk >= 17179869184.0) return FALCON_ERR_UNSUPPORTED;
  const falcon::DeltaDecodeArgs a{nseq, heads, dk, dv, dtype, S, q, k, v, beta, log_a, o};
  return finish_launch(falcon::launch_delta_decode(a, (hipStream_t)stream));
}

namespace {

// What rotary_in and its gradient check of the rotation.
bool rotation_ok(const long long* positions, const double* freqs, int rot, int pairs, float scale,
                 int normalize, int dk) {
  return positions && freqs && ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(freqs)) & 7u) == 0 &&
         rot >= 2 && rot <= dk && rot % 2 == 0 && (pairs == FALCON_PAIRS_HALF || pairs == FALCON_PAIRS_NEIGHBOURS) &&
         isfinite(scale) && (normalize == 0 || normalize == 1);
}

}  // namespace

FALCON_EXPORT int falcon_rotary_in(int batch, int heads, int seqlen, int dk, int dv, int dtype,
                                   const void* q_in, long long ld_q, const void* k_in, long long ld_k,
                                   const void* v_in, long long ld_v, const long long* positions,
                                   const double* freqs, int rot, int pairs, float scale, int normalize,
                                   float eps, void* q, void* k, void* v, void* stream) {
  size_t N, es;
  int st = check_sizes(batch, heads, seqlen, dk, dv, dtype, &N, &es);
  if (st != FALCON_OK) return st;
  if (!finite_nonneg(eps)) return FALCON_ERR_INVALID_ARG;
  if (!q_in || !k_in || !q || !k || (v_in == nullptr) != (v == nullptr))
    return FALCON_ERR_INVALID_ARG;
  if (!rotation_ok(positions, freqs, rot, pairs, scale, normalize, dk)) return FALCON_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v};
  if (!all_aligned16(ptrs)) return FALCON_ERR_INVALID_ARG;
  Rows rq, rk, rv;
  if (check_rows(q_in, ld_q, heads, dk, N, es, &rq) || check_rows(k_in, ld_k, heads, dk, N, es, &rk) ||
      check_rows(v_in, ld_v, heads, dv, N, es, &rv))
    return FALCON_ERR_INVALID_ARG;
  const Range outs[] = {{q, N * heads * dk * es}, {k, N * heads * dk * es}, {v, N * heads * dv * es}};
  const Range ins[] = {hull(rq), hull(rk), hull(rv), {positions, N * 8}, {freqs, (size_t)rot * 4}};
  if (any_overlap(outs, ins)) return FALCON_ERR_INVALID_ARG;
  if (!supported_dim(dk) || !supported_dim(dv) || !norm_heads(heads)) return FALCON_ERR_UNSUPPORTED;
  const falcon::Rotation r{positions, freqs, rot, pairs, scale, normalize};
  const falcon::RotaryInArgs a{batch, heads, seqlen, dk, dv, dtype, r, eps, q_in, (long)ld_q, k_in,
                               (long)ld_k, v_in, (long)ld_v, q, k, v};
  return finish_launch(falcon::launch_rotary_in(a, (hipStream_t)stream));
}

FALCON_EXPORT int falcon_rotary_in_bwd(int batch, int heads, int seqlen, int dk, int dv, int dtype,
                                       const void* q_in, long long ld_q, const void* k_in, long long ld_k,
                                       const long long* positions, const double* freqs, int rot, int pairs,
                                       float scale, int normalize, float eps, const float* dq,
                                       const float* dk_, const float* dv_, void* dq_in, long long ld_dq,
                                       void* dk_in, long long ld_dk, void* dv_in, long long ld_dv,
                                       void* stream) {
  size_t N, es;
  int st = check_sizes(batch, heads, seqlen, dk, dv, dtype, &N, &es);
  if (st != FALCON_OK) return st;
  if (!finite_nonneg(eps)) return FALCON_ERR_INVALID_ARG;
  if (!q_in || !k_in || !dq || !dk_ || !dq_in || !dk_in || (dv_ == nullptr) != (dv_in == nullptr))
    return FALCON_ERR_INVALID_ARG;
  if (!rotation_ok(positions, freqs, rot, pairs, scale, normalize, dk)) return FALCON_ERR_INVALID_ARG;
  const void* ptrs[] = {dq, dk_, dv_};
  if (!all_aligned16(ptrs)) return FALCON_ERR_INVALID_ARG;
  Rows rq, rk, oq, ok, ov;
  if (check_rows(q_in, ld_q, heads, dk, N, es, &rq) || check_rows(k_in, ld_k, heads, dk, N, es, &rk) ||
      check_rows(dq_in, ld_dq, heads, dk, N, es, &oq) || check_rows(dk_in, ld_dk, heads, dk, N, es, &ok) ||
      check_rows(dv_in, ld_dv, heads, dv, N, es, &ov))
    return FALCON_ERR_INVALID_ARG;
  const Rows outs[] = {oq, ok, ov};
  const Range ins[] = {hull(rq), hull(rk), {dq, N * heads * dk * 4}, {dk_, N * heads * dk * 4},
                       {dv_, N * heads * dv * 4}, {positions, N * 8}, {freqs, (size_t)rot * 4}};
  for (int i = 0; i < 3; ++i) {
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return FALCON_ERR_INVALID_ARG;
    for (const Range& r : ins)
      if (overlap(hull(outs[i]), r)) return FALCON_ERR_INVALID_ARG;
  }
  if (!supported_dim(dk) || !supported_dim(dv) || !norm_heads(heads)) return FALCON_ERR_UNSUPPORTED;
  const falcon::Rotation r{positions, freqs, rot, pairs, scale, normalize};
  const falcon::RotaryInBwdArgs a{batch, heads, seqlen, dk, dv, dtype, r, eps, q_in, (long)ld_q, k_in,
                                  (long)ld_k, dq, dk_, dv_, dq_in, (long)ld_dq, dk_in, (long)ld_dk,
                                  dv_in, (long)ld_dv};
  return finish_launch(falcon::launch_rotary_in_bwd(a, (hipStream_t)stream));
}
