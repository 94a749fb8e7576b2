// Host helpers that the entry points of the C ABI share (defined in api.cpp).
#pragma once

#include "zero_dp_internal.h"

namespace zdp {

// Set the thread's error text and return `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char* what);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// What the launches need to know of a device, found once per device.
struct DeviceInfo {
  bool gfx950;
  size_t batch_lds;  // dynamic LDS per block of the batched update schedule
};

int check_device(DeviceInfo* info = nullptr);

int check_workspace(const void* ws, size_t have);

// Workspace: per-group level-2 partials, then the block partials of the latest launch.
inline double* level2_of(void* ws, int32_t g) { return static_cast<double*>(ws) + static_cast<int64_t>(g) * kFoldBlocks; }
inline double* scratch_of(void* ws) { return reinterpret_cast<double*>(static_cast<char*>(ws) + kHeaderBytes); }

hipError_t fold_into(void* ws, int32_t g, int64_t blocks, hipStream_t s);

}  // namespace zdp
