// Drives the host side of a layer's operators (layer_api.cpp) under the address
// and undefined-behaviour sanitizers: the argument checks of every call at their
// edges, and the sizes that have nothing to do. No launch may be reached.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../zero_dp_partitioned_amd/csrc/layer_internal.h"

namespace zdp {
static hipError_t never_layer(const char* what) {
  fprintf(stderr, "host checks: %s reached a launch\n", what);
  abort();
}
hipError_t launch_norm(const NormArgs&, int32_t, hipStream_t) { return never_layer("norm"); }
hipError_t launch_norm_grad(const NormGradArgs&, int32_t, hipStream_t) { return never_layer("norm gradient"); }
hipError_t launch_dropout(const DropoutArgs&, int32_t, hipStream_t) { return never_layer("dropout"); }
hipError_t launch_gated(const GatedArgs&, int32_t, hipStream_t) { return never_layer("gated product"); }
hipError_t launch_gated_grad(const GatedGradArgs&, int32_t, hipStream_t) { return never_layer("gated gradient"); }
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
  int64_t* const c = reinterpret_cast<int64_t*>(buf);
  const size_t ws = zero_workspace_bytes(1);
  const int64_t big[] = {INT64_MAX, INT64_MAX - 3, INT64_MAX / 2, INT64_MAX / 4 + 1, int64_t{1} << 61};
  for (int64_t v : big) {
    EXPECT(zero_layer_norm(p, ZERO_DT_F32, v, 8, 8, f, f, ZERO_DT_F32, 1e-5, p, 8, f, f, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_layer_norm(p, ZERO_DT_F32, 4, 8, v, f, f, ZERO_DT_F32, 1e-5, p, 8, f, f, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_layer_norm(p, ZERO_DT_F32, 4, v, v, f, f, ZERO_DT_F32, 1e-5, p, v, f, f, nullptr), ZERO_ERR_UNSUPPORTED);
    EXPECT(zero_layer_norm_backward(p, 8, p, 8, ZERO_DT_F16, v, 8, p, ZERO_DT_F16, f, f, nullptr, 0, p, 8, nullptr, nullptr, 0,
                                    0, nullptr, 0, nullptr),
           ZERO_ERR_INVALID_ARG);
    EXPECT(zero_layer_norm_backward(p, 8, p, 8, ZERO_DT_F16, 4, 8, p, ZERO_DT_F16, f, f, p, v, p, 8, p, p, ZERO_DT_F32, 1, p,
                                    ws, nullptr),
           ZERO_ERR_INVALID_ARG);
    EXPECT(zero_dropout(p, ZERO_DT_BF16, v, 8, 8, nullptr, 0, p, 8, 0.5, 1, 2, nullptr, 0, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_dropout(p, ZERO_DT_BF16, 1, v, v, nullptr, 0, p, v, 0.5, 1, 2, nullptr, INT64_MAX - 5, nullptr),
           ZERO_ERR_INVALID_ARG);
    EXPECT(zero_dropout(p, ZERO_DT_F32, 4, 4, 4, p, v, p, 4, 0.5, 1, 2, c, 0, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_gated_product(p, ZERO_DT_F16, v, 8, 8, p, p, 8, 8, 0, p, 8, nullptr, nullptr, 0, nullptr), ZERO_ERR_UNSUPPORTED);
    EXPECT(zero_gated_product(p, ZERO_DT_F16, 4, 8, v, p, p, 8, 8, 0, p, 8, nullptr, nullptr, 0, nullptr), ZERO_ERR_INVALID_ARG);
    EXPECT(zero_gated_product_backward(p, v, p, ZERO_DT_F16, 4, 8, 8, p, p, 8, 8, 0, p, p, 8, p, p, 8, p, 8, p, p, 8,
                                       ZERO_DT_F32, 0, p, ws, nullptr),
           ZERO_ERR_INVALID_ARG);
    EXPECT(zero_gated_product_backward(p, 8, p, ZERO_DT_F16, 4, 8, 8, p, p, 8, 8, 0, p, p, 8, p, p, 8, p, 8, p, p, v,
                                       ZERO_DT_F32, 0, p, ws, nullptr),
           ZERO_ERR_INVALID_ARG);
  }
  // probabilities and epsilons at their edges
  const double bad_p[] = {-0.1, 1.0, 1.0 - 0x1p-40, 1e300, -INFINITY, INFINITY, NAN};
  for (double v : bad_p)
    EXPECT(zero_dropout(p, ZERO_DT_F32, 2, 4, 4, nullptr, 0, p, 4, v, 1, 2, nullptr, 0, nullptr), ZERO_ERR_INVALID_ARG);
  const double bad_eps[] = {-1e-30, -INFINITY, INFINITY, NAN};
  for (double v : bad_eps)
    EXPECT(zero_layer_norm(p, ZERO_DT_F32, 2, 4, 4, f, nullptr, ZERO_DT_F32, v, p, 4, nullptr, nullptr, nullptr),
           ZERO_ERR_INVALID_ARG);
  EXPECT(zero_dropout(p, ZERO_DT_F32, 2, 4, 4, nullptr, 0, p, 4, 0.5, 1, 2, nullptr, INT64_MIN, nullptr), ZERO_ERR_INVALID_ARG);
  // nothing to do
  EXPECT(zero_layer_norm(nullptr, ZERO_DT_F16, 0, 8, 8, nullptr, nullptr, ZERO_DT_F16, 0.0, nullptr, 8, nullptr, nullptr, nullptr),
         ZERO_OK);
  EXPECT(zero_layer_norm_backward(nullptr, 0, nullptr, 0, ZERO_DT_F16, 5, 0, nullptr, ZERO_DT_F16, nullptr, nullptr, nullptr, 0,
                                  nullptr, 0, nullptr, nullptr, 0, 0, nullptr, 0, nullptr),
         ZERO_OK);
  EXPECT(zero_dropout(nullptr, ZERO_DT_F32, 0, INT64_MAX, INT64_MAX, nullptr, 0, nullptr, INT64_MAX, 0.0, 0, 0, nullptr,
                      INT64_MAX, nullptr),
         ZERO_OK);
  EXPECT(zero_gated_product(nullptr, ZERO_DT_BF16, 0, 8, 8, nullptr, nullptr, 0, 8, 4, nullptr, 0, nullptr, nullptr, 0, nullptr),
         ZERO_OK);
  if (failures == 0) printf("layer host checks: ok\n");
  return failures != 0;
}
