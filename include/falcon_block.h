/*
 * falcon_block.h - C interface of libfalcon_block: the gated delta rule and rotary
 * positions at a block's entry, next to the update rules and norms of falcon.h, on
 * AMD Instinct MI355X (gfx950).  Types, status codes, layouts, ownership and
 * determinism are falcon.h's; a library of its own, so that libfalcon's interface
 * and version stay what they are.
 */
#ifndef FALCON_BLOCK_H
#define FALCON_BLOCK_H

#include "falcon.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The gated delta rule, per (batch, head), t = 1..L:
 *   S_t = a_t S_{t-1} + u_t k_t^T,   u_t = beta_t (v_t - a_t S_{t-1} k_t),
 *   o_t = S_t q_t,                   a_t = exp(log_a_t)
 * that is S_t = a_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T: Falcon-1's
 * squared-error step with a decay of its own in place of 1 - eta lambda, the same step's
 * key, and a step size that is not divided by the key's energy.
 *   beta     [batch, heads, L] float32, finite
 *   log_a    [batch, heads, L] float32, or NULL (a = 1).  A token whose decay is below 2^-126, the
 *            smallest normal float32 (-inf, and any log decay below about -87.34), is a reset: its
 *            decay counts as 0, and a new sequence starts at it.  (In _fwd_chunk and _bwd_chunk a
 *            product of several tokens' decays counts as 0 below 2^-126, too, and is off by up to
 *            2^-134: below 2^-110 it keeps fewer bits than a float32.)
 * (beta, log_a, dbeta, dlog_a 4-byte aligned, every other pointer 16)
 *
 * falcon_gated_delta_fwd_chunk - a sequence, in chunks of 64 tokens
 *   q, k, v, S0, o, S_out   as falcon_fwd_chunk (S0, S_out may be NULL; S_out may equal
 *            S0); bf16 or fp32 inputs, dk, dv in {16, 32, 64, 128}, any L >= 1
 *   workspace  falcon_gated_delta_fwd_workspace_bytes(...) bytes of device memory, 16-byte
 *            aligned, overlapping no other argument; it serves one call at a time
 * The recurrence to float32 rounding for keys and steps that keep it stable
 * (0 <= beta_t |k_t|^2 <= 2 and log_a <= 0: unit keys and a sigmoid's beta are): products
 * run on bf16 matrix cores with float32 operands in three bf16 parts, decays as differences of
 * float64 sums.  Outside of that range S may grow by a factor a token, and so do its
 * roundings; a growth that float32 does not hold gives infinities and NaN, also of a state
 * of zeros (a long sequence of few heads is walked in segments, each of which forms the
 * matrix that it applies).  A NaN or an infinity reaches the outputs that read it, o of its token and of
 * later ones and S_out, and no others: rows of padding behind a sequence may hold
 * anything.  (A reset does not clear it: 0 * NaN.  float32 inputs and states beyond bf16's
 * 3.39e38 count as infinite.  Segments that hold one, or start
 * from one, are walked again token by token, which takes many times as long.)
 * FALCON_ERR_UNSUPPORTED from batch * heads * max(dk, dv) * (L + 63) / 64 = 2^31 on, and where a
 * launch would have 2^32 work-items: 12 dv for each (batch, head), whose number counts as the next
 * multiple of 8, or 64 for each 64-token chunk (four chunks together).
 *
 * falcon_gated_delta_bwd_chunk - gradients of sum <dO, o> + <dS_L, S_L>
 *   q, k, v, beta, log_a, S0, dtype   as the forward's
 *   dO       [batch, heads, L, dv] float32
 *   dS_L     [batch, heads, dv, dk] float32, or NULL
 *   dq, dk_out, dv_out   [batch, heads, L, dk / dk / dv] float32
 *   dbeta    [batch, heads, L] float32
 *   dlog_a   [batch, heads, L] float32, or NULL; needs log_a.  0 at a reset, and before one
 *            nothing of what lies behind it.  A difference of sums: its error is float32
 *            rounding of q . dq and v . dv of the tokens from it to its 64-token chunk's end,
 *            not of itself
 *   dS0      [batch, heads, dv, dk] float32, or NULL (with S0 NULL: the gradient of the
 *            zero state)
 *   workspace  falcon_gated_delta_bwd_workspace_bytes(...) bytes, 16-byte aligned
 * Here a NaN or an infinity in a token also reaches gradients that do not depend on it, of its
 * 64-token chunk.  Rows of padding have to be finite.  Outputs and workspace overlap no other
 * argument.  Sizes as the forward's, with 512 work-items for each (batch, head) at dv = 32, 384 at
 * dv = 16, and 256 for each 64-token chunk.
 *
 * falcon_gated_delta_decode_step - one token for serving: S [nseq, heads, dv, dk]
 * float32 updated in place, q, k [nseq, heads, dk], v [nseq, heads, dv], beta and log_a
 * [nseq, heads] (log_a or NULL), o [nseq, heads, dv] float32.  No argument may overlap
 * another.  nseq * heads * dk * dv < 2^34 (FALCON_ERR_UNSUPPORTED from there on).
 */
unsigned long long falcon_gated_delta_fwd_workspace_bytes(int batch, int heads, int seqlen, int dk,
                                                          int dv, int dtype);
int falcon_gated_delta_fwd_chunk(int batch, int heads, int seqlen, int dk, int dv, int dtype,
                                 const void* q, const void* k, const void* v, const float* beta,
                                 const float* log_a, const float* S0, float* o, float* S_out,
                                 void* workspace, unsigned long long workspace_bytes, void* stream);
unsigned long long falcon_gated_delta_bwd_workspace_bytes(int batch, int heads, int seqlen, int dk,
                                                          int dv, int dtype);
int falcon_gated_delta_bwd_chunk(int batch, int heads, int seqlen, int dk, int dv, int dtype,
                                 const void* q, const void* k, const void* v, const float* beta,
                                 const float* log_a, const float* S0, const float* dO,
                                 const float* dS_L, float* dq, float* dk_out, float* dv_out,
                                 float* dbeta, float* dlog_a, float* dS0, void* workspace,
                                 unsigned long long workspace_bytes, void* stream);
int falcon_gated_delta_decode_step(int nseq, int heads, int dk, int dv, int dtype, float* S,
                                   const void* q, const void* k, const void* v, const float* beta,
                                   const float* log_a, float* o, void* stream);

/*
 * Rotary positions at a block's entry: falcon_norm_in with the first `rot` columns of every
 * q and k row turned, in pairs, by an angle proportional to the token's position.
 *
 * falcon_rotary_in - per token (b, t), head and pair i < rot / 2
 *   x = q_in / sqrt(|q_in|^2 + eps)      (x = q_in with normalize = 0; k likewise)
 *   angle = positions[b, t] * freqs[i]
 *   (y_first, y_second) = scale * (x_first cos - x_second sin, x_second cos + x_first sin)
 * the columns from rot on pass, v = v_in.
 *   q_in, k_in, v_in   token-major with strides, as falcon_norm_in
 *   positions          [batch, L] 64-bit integers, |position| < 2^53
 *   freqs              [rot / 2] float64, radians a token; angles are reduced to float32
 *                      rounding at every position
 *   rot                even, 2 <= rot <= dk
 *   pairs              FALCON_PAIRS_HALF (columns i and i + rot / 2) or
 *                      FALCON_PAIRS_NEIGHBOURS (2 i and 2 i + 1)
 *   scale              finite; of the turned columns
 *   q, k, v            head-major, contiguous; v_in and v may both be NULL
 *
 * falcon_rotary_in_bwd - its gradient, arguments as falcon_norm_in_bwd: dq and dk turned
 * back and scaled, then the norm's gradient (with normalize = 0 none).
 *
 * Sizes, errors and rounding as the norms of falcon.h.
 */
#define FALCON_PAIRS_HALF 0
#define FALCON_PAIRS_NEIGHBOURS 1
int falcon_rotary_in(int batch, int heads, int seqlen, int dk, int dv, int dtype, const void* q_in,
                     long long ld_q, const void* k_in, long long ld_k, const void* v_in,
                     long long ld_v, const long long* positions, const double* freqs, int rot,
                     int pairs, float scale, int normalize, float eps, void* q, void* k, void* v,
                     void* stream);
int falcon_rotary_in_bwd(int batch, int heads, int seqlen, int dk, int dv, int dtype,
                         const void* q_in, long long ld_q, const void* k_in, long long ld_k,
                         const long long* positions, const double* freqs, int rot, int pairs,
                         float scale, int normalize, float eps, const float* dq, const float* dk_,
                         const float* dv_, void* dq_in, long long ld_dq, void* dk_in,
                         long long ld_dk, void* dv_in, long long ld_dv, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FALCON_BLOCK_H */
