// Drives the host side of the microscaled 4-bit calls (mx_api.cpp) under the
// address and undefined-behaviour sanitizers: the argument checks of every
// call at their edges, and the sizes that have nothing to do. No launch may be
// reached.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "../../zero_dp_partitioned_amd/csrc/mx_internal.h"

namespace zdp {
static hipError_t never_mx(const char* what) {
  fprintf(stderr, "host checks: %s reached a launch\n", what);
  abort();
}
hipError_t launch_mx_quantize(const MxQuantArgs&, int32_t, hipStream_t) { return never_mx("quantise"); }
hipError_t launch_mx_widen(const MxWidenArgs&, int32_t, hipStream_t) { return never_mx("widen"); }
hipError_t launch_mx_reduce(const MxReduceArgs&, hipStream_t, int*) { return never_mx("4-bit average"); }
hipError_t launch_mx_product(const MxProductArgs&, int32_t, hipStream_t) { return never_mx("product"); }
}  // namespace zdp

static int failures = 0;
#define EXPECT(rc, want)                                                              \
  do {                                                                                \
    const int got = (rc);                                                             \
    if (got != (want)) {                                                              \
      printf("line %d: %d, expected %d (%s)\n", __LINE__, got, want, zero_last_error()); \
      ++failures;                                                                     \
    }                                                                                 \
  } while (0)

int main() {
  alignas(256) static uint8_t buf[4096];
  uint8_t* const p = buf;
  float* const f = reinterpret_cast<float*>(buf);
  const int64_t big[] = {INT64_MAX, INT64_MAX - 31, INT64_MAX / 2, INT64_MAX / 16, int64_t{1} << 60};
  for (int64_t v : big) {
    EXPECT(zero_mx_quantize(f, ZERO_DT_F32, v, 32, 32, p, p, 1, nullptr, nullptr, 0, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_mx_quantize(f, ZERO_DT_F32, 2, v, v, p, p, v, nullptr, nullptr, 0, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_mx_quantize(f, ZERO_DT_BF16, 16, 32, v, p, p, 1, nullptr, nullptr, 0, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_mx_quantize(f, ZERO_DT_F16, 64, 2, 2, nullptr, nullptr, 0, p, p, v, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_mx_dequantize(p, p, 2, 32, v, f, ZERO_DT_F32, 32, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_mx_dequantize(p, p, v, 32, 1, f, ZERO_DT_F32, 32, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_mx_product(p, p, v, p, p, 1, 2, 2, 1, f, ZERO_DT_F32, 2, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_mx_product(p, p, 1, p, p, 1, v, 2, 1, f, ZERO_DT_F32, 2, nullptr), ZERO_ERR_UNSUPPORTED);
    EXPECT(zero_mx_product(p, p, 1, p, p, 1, 2, 2, v, f, ZERO_DT_F32, 2, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_mx_cast_writeback(f, 32, p, p, v - v % 32 + 1, nullptr), ZERO_ERR_INVALID_ARG);
  }
  EXPECT(zero_mx_quantize(nullptr, ZERO_DT_F32, 0, 7, 7, nullptr, nullptr, 0, nullptr, nullptr, 0, nullptr), ZERO_OK);
  EXPECT(zero_mx_dequantize(nullptr, nullptr, 7, 0, 0, nullptr, ZERO_DT_F16, 0, nullptr), ZERO_OK);
  EXPECT(zero_mx_product(nullptr, nullptr, 4, p, p, 4, 0, 3, 4, nullptr, ZERO_DT_BF16, 3, nullptr), ZERO_OK);
  EXPECT(zero_mx_cast_writeback(nullptr, 0, nullptr, nullptr, 32, nullptr), ZERO_OK);

  // copies: up to the inline table any pointers, beyond it equal spacing, up to the maximum
  std::vector<const void*> codes(ZERO_MAX_REPLICAS + 1), scales(ZERO_MAX_REPLICAS + 1);
  for (int32_t r = 0; r <= ZERO_MAX_REPLICAS; ++r) {
    codes[r] = reinterpret_cast<const void*>(uintptr_t{1 << 20} + 64 * static_cast<uintptr_t>(r));
    scales[r] = reinterpret_cast<const void*>(uintptr_t{1 << 20} + 3 * static_cast<uintptr_t>(r));
  }
  const size_t ws = zero_workspace_bytes(1);
  zero_step_state* const st = reinterpret_cast<zero_step_state*>(buf);
  EXPECT(zero_mx_reduce_grad_segment(codes.data(), scales.data(), ZERO_MAX_REPLICAS + 1, 64, f, buf, ws, 0, st, nullptr),
         ZERO_ERR_UNSUPPORTED);
  for (int32_t n_d : {65, 100, ZERO_MAX_REPLICAS}) {
    std::vector<const void*> odd(codes);
    odd[n_d - 1] = codes[0];
    EXPECT(zero_mx_reduce_grad_segment(odd.data(), scales.data(), n_d, 64, f, buf, ws, 0, st, nullptr),
           ZERO_ERR_UNSUPPORTED);
    EXPECT(zero_mx_reduce_grad_segment(codes.data(), odd.data(), n_d, 64, f, buf, ws, 0, st, nullptr),
           ZERO_ERR_UNSUPPORTED);
  }
  for (int32_t n_d : {1, 64, ZERO_MAX_REPLICAS}) {
    std::vector<const void*> bad(codes);
    bad[n_d - 1] = static_cast<const uint8_t*>(codes[n_d - 1]) + 8;
    EXPECT(zero_mx_reduce_grad_segment(bad.data(), scales.data(), n_d, 64, f, buf, ws, 0, st, nullptr),
           ZERO_ERR_ALIGNMENT);
    bad[n_d - 1] = nullptr;
    EXPECT(zero_mx_reduce_grad_segment(bad.data(), scales.data(), n_d, 64, f, buf, ws, 0, st, nullptr),
           ZERO_ERR_INVALID_ARG);
  }
  if (failures) return 1;
  printf("mx host checks: ok\n");
  return 0;
}
