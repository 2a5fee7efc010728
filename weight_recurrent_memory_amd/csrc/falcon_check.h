// falcon_check.h - checks of arguments shared by the C layers (falcon_api.cpp and
// falcon_block_api.cpp); each includes it once.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "falcon.h"

#define FALCON_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool supported_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

bool finite_nonneg(float x) { return isfinite(x) && x >= 0.0f; }

struct Range {
  const void* p;
  size_t bytes;
};

bool overlap(Range a, Range b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

int finish_launch(hipError_t e) { return e == hipSuccess ? FALCON_OK : FALCON_ERR_HIP; }

// A token-major argument: N rows of `width` bytes, `pitch` bytes apart.
struct Rows {
  const void* p;
  size_t n, width, pitch;
};

Range hull(const Rows& r) { return Range{r.p, r.p ? (r.n - 1) * r.pitch + r.width : 0}; }

// Whether two token-major arguments share a byte.  Rows of one pitch may
// interleave (views of one fused buffer); other hulls that meet count as shared.
bool overlap(const Rows& a, const Rows& b) {
  if (!overlap(hull(a), hull(b))) return false;
  if (a.pitch != b.pitch) return true;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const size_t d = pb >= pa ? (pb - pa) % a.pitch : (a.pitch - (pa - pb) % a.pitch) % a.pitch;
  return d < a.width || a.pitch - d < b.width;
}

// Sizes common to the calls below; fills N (tokens) and es (element size).
int check_sizes(int batch, int heads, int seqlen, int d0, int d1, int dtype, size_t* N, size_t* es) {
  if (batch < 1 || heads < 1 || seqlen < 1 || d0 < 1 || d1 < 1) return FALCON_ERR_INVALID_ARG;
  if (dtype != FALCON_BF16 && dtype != FALCON_F32) return FALCON_ERR_INVALID_ARG;
  if ((double)batch * heads * seqlen * (d0 > d1 ? d0 : d1) > 1099511627776.0)
    return FALCON_ERR_INVALID_ARG;  // 2^40 elements
  if ((double)batch * seqlen >= 2147483648.0) return FALCON_ERR_INVALID_ARG;
  *N = (size_t)batch * seqlen;
  *es = dtype == FALCON_BF16 ? 2 : 4;
  return FALCON_OK;
}

// One token-major argument's pointer and stride.
int check_rows(const void* p, long long ld, int heads, int d, size_t N, size_t es, Rows* out) {
  *out = Rows{nullptr, 1, 0, 1};
  if (!p) return FALCON_OK;
  if (!aligned16(p) || ld < (long long)heads * d || ld > (1ll << 40) || (ld * (long long)es) % 16 != 0)
    return FALCON_ERR_INVALID_ARG;
  if ((double)N * (double)ld > 4398046511104.0) return FALCON_ERR_INVALID_ARG;  // 2^42 elements
  *out = Rows{p, N, (size_t)heads * d * es, (size_t)ld * es};
  return FALCON_OK;
}

// Outputs against each other and against the inputs (null ones take no part).
template <int NO, int NI>
bool any_overlap(const Range (&outs)[NO], const Range (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return true;
  }
  return false;
}

template <int N>
bool all_aligned16(const void* const (&ptrs)[N]) {
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return false;
  return true;
}

// Heads of the norms: a workgroup's rows, up to 16 tokens of every head, are counted in 32 bits.
bool norm_heads(int heads) { return heads < (1 << 27); }

// Log decays are read and written one by one.
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
