// Host-side check of the norms' and the gated recurrence's entry points under
// AddressSanitizer and UndefinedBehaviorSanitizer (built and run by
// tests/test_host_sanitize_block.py on a machine without a GPU): argument checks, the
// overlap arithmetic of interleaved rows, workspace sizes and the plans of large calls.
// Pointers are stand-in addresses 2^44 bytes apart, which this layer compares and offsets
// and never reads through; a well-formed call gets as far as its first launch, which fails
// for want of a device (FALCON_ERR_HIP).
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <limits>

#include "falcon.h"

// The kernels' code objects are not part of this build: no launch gets as far as one.
extern "C" {
alignas(4096) extern const unsigned char no_device_code[4096] = {0};
}

namespace {

int g_checks = 0, g_failures = 0;

void expect(const char* what, long long got, long long want) {
  ++g_checks;
  if (got == want) return;
  ++g_failures;
  std::printf("FAIL %s: got %lld, want %lld\n", what, got, want);
}

template <typename T = void>
T* far(int i, long long bytes = 0) {
  return reinterpret_cast<T*>((static_cast<uintptr_t>(i) + 1) * (1ull << 44) + static_cast<uintptr_t>(bytes));
}

constexpr int kOk = FALCON_ERR_HIP;          // all checks passed, no device
constexpr int kBad = FALCON_ERR_INVALID_ARG, kNo = FALCON_ERR_UNSUPPORTED;
const int kDims[] = {16, 32, 64, 128};

struct Shape {
  int batch, heads, seqlen;
};

// ------------------------------------------------------------------ norms

// q, k, v as views of one buffer of rows `ld` elements apart
int norm_in(Shape s, int dk, int dv, int dtype, long long ld, bool values) {
  const long long es = dtype == FALCON_BF16 ? 2 : 4, wk = (long long)s.heads * dk * es;
  return falcon_norm_in(s.batch, s.heads, s.seqlen, dk, dv, dtype, far(0), ld, far(0, wk), ld,
                        values ? far(0, 2 * wk) : nullptr, ld, 1e-6f, far(1), far(2),
                        values ? far(3) : nullptr, nullptr);
}
// shift: bytes that the k rows of the fused output lie off their place
int norm_in_bwd(Shape s, int dk, int dv, int dtype, long long ld, bool values, long long shift = 0) {
  const long long es = dtype == FALCON_BF16 ? 2 : 4, wk = (long long)s.heads * dk * es;
  return falcon_norm_in_bwd(s.batch, s.heads, s.seqlen, dk, dv, dtype, far(0), ld, far(0, wk), ld, 1e-6f,
                            far<float>(1), far<float>(2), values ? far<float>(3) : nullptr, far(4), ld,
                            far(4, wk + shift), ld, values ? far(4, 2 * wk) : nullptr, ld, nullptr);
}
int norm_out(Shape s, int dv, int dtype, long long ld, bool gate, bool residual, bool in_place) {
  return falcon_norm_out(s.batch, s.heads, s.seqlen, dv, dtype, far<float>(0), far<float>(1),
                         gate ? far(2) : nullptr, ld, FALCON_GATE_SILU, residual ? far(3) : nullptr, ld, 0.5f,
                         1e-6f, in_place ? far(3) : far(4), ld, nullptr);
}
int norm_out_bwd(Shape s, int dv, int dtype, long long ld, bool gate, long long short_by = 0) {
  const unsigned long long need = falcon_norm_out_bwd_workspace_bytes(s.batch, s.seqlen, dv);
  return falcon_norm_out_bwd(s.batch, s.heads, s.seqlen, dv, dtype, far<float>(0), far<float>(1),
                             gate ? far(2) : nullptr, ld, FALCON_GATE_SIGMOID, 0.5f, 1e-6f, far(3), ld,
                             far<float>(4), gate ? far(5) : nullptr, ld, far<float>(6), far(7),
                             need - (unsigned long long)short_by, nullptr);
}

void norm_cases() {
  const Shape shapes[] = {{1, 1, 1}, {7, 3, 1}, {2, 5, 4099}, {1, 1, std::numeric_limits<int>::max()},
                          {1, (1 << 27) - 1, 1}, {std::numeric_limits<int>::max(), 1, 1}, {1 << 15, 2, (1 << 16) - 1}};
  for (const Shape& s : shapes)
    for (int dk : kDims)
      for (int dv : kDims)
        for (int dtype = 0; dtype < 2; ++dtype) {
          const long long ld = (long long)s.heads * (2 * dk + dv) + 16;
          // the sizes above stay under 2^40 elements and 2^42 with their rows' distance
          expect("norm_in", norm_in(s, dk, dv, dtype, ld, true), kOk);
          expect("norm_in without v", norm_in(s, dk, dv, dtype, ld, false), kOk);
          expect("norm_in_bwd", norm_in_bwd(s, dk, dv, dtype, ld, true), kOk);
          expect("norm_in_bwd without v", norm_in_bwd(s, dk, dv, dtype, ld, false), kOk);
          if ((double)s.batch * s.seqlen > 1)
            expect("norm_in_bwd, rows that meet", norm_in_bwd(s, dk, dv, dtype, ld, true, 16), kBad);
          expect("norm_out", norm_out(s, dv, dtype, ld, true, true, false), kOk);
          expect("norm_out in place", norm_out(s, dv, dtype, ld, false, true, true), kOk);
          expect("norm_out_bwd", norm_out_bwd(s, dv, dtype, ld, true), kOk);
          expect("norm_out_bwd without a gate", norm_out_bwd(s, dv, dtype, ld, false), kOk);
          expect("norm_out_bwd, short workspace", norm_out_bwd(s, dv, dtype, ld, true, 1), kBad);
        }
  const Shape s{2, 3, 8};
  expect("norm_in, rows off 16 bytes", norm_in(s, 64, 64, 0, 580, true), kBad);
  expect("norm_in, rows too near", norm_in(s, 64, 64, 0, 191, true), kBad);
  expect("norm_in, rows too far", norm_in(s, 64, 64, 0, std::numeric_limits<long long>::max() / 16 * 8, true), kBad);
  expect("norm_in, rows backward", norm_in(s, 64, 64, 0, std::numeric_limits<long long>::min(), true), kBad);
  expect("norm_in, tokens", norm_in({1 << 16, 1, 1 << 15}, 64, 64, 0, 192, true), kBad);
  expect("norm_in, heads", norm_in({1, 1 << 27, 1}, 16, 16, 0, 3ll << 31, true), kNo);
  expect("norm_in, size", norm_in(s, 48, 64, 0, 576, true), kNo);
  expect("workspace of no size", (long long)falcon_norm_out_bwd_workspace_bytes(1, 1, 48), 0);
  expect("workspace of too many tokens", (long long)falcon_norm_out_bwd_workspace_bytes(1 << 16, 1 << 15, 16), 0);
}

// ------------------------------------------------------- gated recurrence

int gated_fwd(Shape s, int dk, int dv, int dtype, bool gates, bool state, bool cut) {
  const unsigned long long need = falcon_gated_fwd_workspace_bytes(s.batch, s.heads, s.seqlen, dk, dv, dtype);
  return falcon_gated_fwd_chunk(s.batch, s.heads, s.seqlen, dk, dv, dtype, far(0), far(1), far(2),
                                gates ? far<float>(3, 4) : nullptr, state ? far<float>(4) : nullptr, far<float>(5),
                                state ? far<float>(4) : nullptr, cut ? far(6) : nullptr, cut ? need : 0, nullptr);
}
int gated_bwd(Shape s, int dk, int dv, int dtype, bool gates, bool state, bool end, long long short_by = 0) {
  const unsigned long long need = falcon_gated_bwd_workspace_bytes(s.batch, s.heads, s.seqlen, dk, dv, dtype);
  return falcon_gated_bwd_chunk(s.batch, s.heads, s.seqlen, dk, dv, dtype, far(0), far(1), far(2),
                                gates ? far<float>(3, 4) : nullptr, state ? far<float>(4) : nullptr, far<float>(5),
                                end ? far<float>(6) : nullptr, far<float>(7), far<float>(8), far<float>(9),
                                gates ? far<float>(10, 8) : nullptr, state ? far<float>(11) : nullptr, far(12),
                                need - (unsigned long long)short_by, nullptr);
}

bool bwd_limit(Shape s, int dk, int dv) {
  const double chains = (double)s.batch * s.heads;
  return chains * (dk > dv ? dk : dv) * ((s.seqlen + 1023.0) / 1024.0) < 67108864.0 &&
         chains * dk * dv < 4294967296.0;
}

void gated_cases() {
  const Shape shapes[] = {{1, 1, 1}, {1, 5, 4099}, {8, 12, 2048}, {64, 16, 700}, {1, 1, std::numeric_limits<int>::max()},
                          {1, 1, std::numeric_limits<int>::max() - 62}, {1, 1, 1 << 30}, {512, 255, 1000},
                          {1 << 11, 1 << 9, 2047}, {2, 3, 1 << 25}};
  for (const Shape& s : shapes)
    for (int dk : kDims)
      for (int dv : kDims)
        for (int dtype = 0; dtype < 2; ++dtype)
          for (int opt = 0; opt < 8; ++opt) {
            const bool fits = (double)s.batch * s.heads * dv < 134217728.0;
            expect("gated_fwd", gated_fwd(s, dk, dv, dtype, opt & 1, opt & 2, opt & 4), fits ? kOk : kNo);
            const bool back = bwd_limit(s, dk, dv);
            expect("gated_bwd", gated_bwd(s, dk, dv, dtype, opt & 1, opt & 2, opt & 4), back ? kOk : kNo);
            if (back && opt == 7)
              expect("gated_bwd, short workspace", gated_bwd(s, dk, dv, dtype, true, true, true, 1), kBad);
          }
  expect("gated_fwd, 2^40 elements and more", gated_fwd({1 << 14, 1 << 13, 1 << 14}, 16, 16, 0, true, true, true), kBad);
  const Shape steps[] = {{1, 1, 1}, {512, 12, 1}, {1 << 15, 31, 1}, {(1 << 20) - 1, 64, 1}};
  for (const Shape& s : steps)
    for (int dk : kDims)
      for (int dv : kDims)
        for (int dtype = 0; dtype < 2; ++dtype)
          expect("gated_decode_step",
                 falcon_gated_decode_step(s.batch, s.heads, dk, dv, dtype, far<float>(0), far(1), far(2), far(3),
                                          far<float>(4, 4), far<float>(5), nullptr),
                 (double)s.batch * s.heads * dk * dv < 17179869184.0 ? kOk : kNo);
  expect("decode, output over the gates",
         falcon_gated_decode_step(2, 3, 64, 64, 0, far<float>(0), far(1), far(2), far(3), far<float>(4), far<float>(4),
                                  nullptr),
         kBad);
}

}  // namespace

int main() {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) == hipSuccess && ndev > 0) {
    std::printf("a GPU is present: this host-only check does not run here\n");
    return 77;
  }
  norm_cases();
  gated_cases();
  std::printf("%d checks, %d failures\n", g_checks, g_failures);
  return g_failures == 0 ? 0 : 1;
}
