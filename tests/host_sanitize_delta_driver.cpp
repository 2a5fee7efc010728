// Host-side check of libfalcon_block's entry points under AddressSanitizer and
// UndefinedBehaviorSanitizer (built and run by tests/test_host_sanitize_delta.py on a machine
// without a GPU): argument checks, workspace sizes, plans and launch shapes up to the
// largest sizes.  Pointers are stand-in addresses that this layer compares and offsets and never
// reads through; a well-formed call gets as far as its first launch, which fails for want
// of a device (FALCON_ERR_HIP).
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>

#include "falcon_block.h"

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
const Shape kShapes[] = {{1, 1, 1}, {2, 3, 77}, {8, 12, 2048}, {1, 4, 32771}, {1, 1, 1 << 24}, {1 << 12, 16, 1}, {4096, 64, 65}};

int forward(Shape s, int dk, int dv, int dtype, unsigned long long ws, bool all = true) {
  return falcon_gated_delta_fwd_chunk(s.batch, s.heads, s.seqlen, dk, dv, dtype, far(0), far(1), far(2), far<float>(3),
                                      all ? far<float>(4) : nullptr, all ? far<float>(5) : nullptr, far<float>(6),
                                      all ? far<float>(5) : nullptr, far(7), ws, nullptr);
}
int backward(Shape s, int dk, int dv, int dtype, unsigned long long ws, bool all = true) {
  return falcon_gated_delta_bwd_chunk(
      s.batch, s.heads, s.seqlen, dk, dv, dtype, far(0), far(1), far(2), far<float>(3), all ? far<float>(4) : nullptr,
      all ? far<float>(5) : nullptr, far<float>(6), all ? far<float>(7) : nullptr, far<float>(8), far<float>(9),
      far<float>(10), far<float>(11), all ? far<float>(12) : nullptr, all ? far<float>(13) : nullptr, far(14), ws,
      nullptr);
}
int rotary(Shape s, int dk, int dv, int dtype, long long ld, int rot, bool values) {
  const long long es = dtype == FALCON_BF16 ? 2 : 4, wk = (long long)s.heads * dk * es;
  return falcon_rotary_in(s.batch, s.heads, s.seqlen, dk, dv, dtype, far(0), ld, far(0, wk), ld,
                          values ? far(0, 2 * wk) : nullptr, ld, far<long long>(1), far<double>(2), rot,
                          FALCON_PAIRS_HALF, 1.0f, 1, 1e-6f, far(3), far(4), values ? far(5) : nullptr, nullptr);
}
int rotary_bwd(Shape s, int dk, int dv, int dtype, long long ld, int rot, bool values) {
  const long long es = dtype == FALCON_BF16 ? 2 : 4, wk = (long long)s.heads * dk * es;
  return falcon_rotary_in_bwd(s.batch, s.heads, s.seqlen, dk, dv, dtype, far(0), ld, far(0, wk), ld, far<long long>(1),
                              far<double>(2), rot, FALCON_PAIRS_NEIGHBOURS, 1.0f, 0, 1e-6f, far<float>(3),
                              far<float>(4), values ? far<float>(5) : nullptr, far(6), ld, far(6, wk), ld,
                              values ? far(6, 2 * wk) : nullptr, ld, nullptr);
}

}  // namespace

int main() {
  int n = 0;
  if (hipGetDeviceCount(&n) == hipSuccess && n > 0) return 77;
  for (const Shape& s : kShapes)
    for (int dk : kDims)
      for (int dv : kDims)
        for (int dtype : {FALCON_BF16, FALCON_F32}) {
          const unsigned long long f = falcon_gated_delta_fwd_workspace_bytes(s.batch, s.heads, s.seqlen, dk, dv, dtype);
          const unsigned long long b = falcon_gated_delta_bwd_workspace_bytes(s.batch, s.heads, s.seqlen, dk, dv, dtype);
          expect("workspace", f > 0 && b > f, 1);
          expect("forward", forward(s, dk, dv, dtype, f), kOk);
          expect("forward, few arguments", forward(s, dk, dv, dtype, f, false), kOk);
          expect("forward, workspace", forward(s, dk, dv, dtype, f - 1), kBad);
          expect("backward", backward(s, dk, dv, dtype, b), kOk);
          expect("backward, few arguments", backward(s, dk, dv, dtype, b, false), kOk);
          expect("backward, workspace", backward(s, dk, dv, dtype, b - 1), kBad);
          const long long ld = (long long)s.heads * (2 * dk + dv);
          for (bool values : {false, true}) {
            expect("rotary", rotary(s, dk, dv, dtype, ld, dk, values), kOk);
            expect("rotary, part", rotary(s, dk, dv, dtype, ld, 6, values), kOk);
            expect("rotary, odd", rotary(s, dk, dv, dtype, ld, 7, values), kBad);
            expect("rotary gradient", rotary_bwd(s, dk, dv, dtype, ld, dk, values), kOk);
            expect("rotary gradient, wide", rotary_bwd(s, dk, dv, dtype, ld, dk + 2, values), kBad);
          }
        }
  for (int dk : kDims)
    for (int dtype : {FALCON_BF16, FALCON_F32}) {
      expect("decode", falcon_gated_delta_decode_step(512, 12, dk, 64, dtype, far<float>(0), far(1), far(2), far(3),
                                                      far<float>(4), far<float>(5), far<float>(6), nullptr), kOk);
      expect("decode, beta", falcon_gated_delta_decode_step(1, 1, dk, 64, dtype, far<float>(0), far(1), far(2), far(3),
                                                            nullptr, nullptr, far<float>(6), nullptr), kBad);
      expect("decode, size", falcon_gated_delta_decode_step(1 << 20, 16, dk, 128, dtype, far<float>(0), far(1),
                                                            far(2), far(3), far<float>(4), nullptr, far<float>(6),
                                                            nullptr), kNo);
    }
  // 2^31 workgroups' worth of value rows and chunks
  expect("forward, size", forward({1 << 14, 1 << 10, 128}, 64, 64, FALCON_BF16, ~0ull >> 8), kNo);
  expect("backward, size", backward({1 << 14, 1 << 10, 128}, 64, 64, FALCON_BF16, ~0ull >> 8), kNo);
  expect("workspace, size", (long long)falcon_gated_delta_fwd_workspace_bytes(1 << 14, 1 << 10, 128, 64, 64, 0), 0);
  // 2^32 work-items of a launch: one call below, one above
  for (int dtype : {FALCON_BF16, FALCON_F32}) {
    expect("forward, value rows", forward({349525, 8, 1}, 16, 128, dtype, ~0ull >> 2), kOk);
    expect("forward, more value rows", forward({349526, 8, 1}, 16, 128, dtype, ~0ull >> 2), kNo);
    expect("forward, chunks", forward({1, 4, (1 << 30) - 64}, 16, 16, dtype, ~0ull >> 2), kOk);
    expect("forward, more chunks", forward({1, 4, (1 << 30) - 63}, 16, 16, dtype, ~0ull >> 2), kNo);
    expect("backward, value rows", backward({1048575, 8, 1}, 16, 32, dtype, ~0ull >> 2), kOk);
    expect("backward, more value rows", backward({1048576, 8, 1}, 16, 32, dtype, ~0ull >> 2), kNo);
    expect("backward, chunks", backward({1, 16, (1 << 26) - 64}, 16, 16, dtype, ~0ull >> 2), kOk);
    expect("backward, more chunks", backward({1, 16, (1 << 26) - 63}, 16, 16, dtype, ~0ull >> 2), kNo);
  }
  std::printf("%d checks, %d failures\n", g_checks, g_failures);
  return g_failures ? 1 : 0;
}
