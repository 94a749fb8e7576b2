// Device helpers of a layer's operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_internal.h"

#pragma clang fp contract(off)

namespace zdp {
namespace {

typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------------
// 16 bytes of values of type DT. Tensors need only be aligned to their
// elements: the 16-byte accesses below work at any such address.
// ------------------------------------------------------------------------

template <int DT>
struct Vec {
  static constexpr int kElem = DT == ZERO_DT_F32 ? 4 : 2;
  static constexpr int kVals = 16 / kElem;
};

// Two fp32 values as 16-bit ones, rounded to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == ZERO_DT_BF16) {
    const f2 x = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf2));
  } else {
    const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<_Float16>(a));
    const uint32_t hi = __builtin_bit_cast(uint16_t, static_cast<_Float16>(b));
    return lo | (hi << 16);
  }
}

template <int DT>
__device__ __forceinline__ float widen16(uint32_t h) {  // of the low 16 bits
  if constexpr (DT == ZERO_DT_BF16) return __uint_as_float(h << 16);
  else return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
}

template <int DT>
__device__ __forceinline__ void widen(const u4 x, float* v) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (DT == ZERO_DT_F32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = __uint_as_float(w[q]);
  } else if constexpr (DT == ZERO_DT_BF16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(w[q] << 16);
      v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = widen16<DT>(w[q]);
      v[2 * q + 1] = widen16<DT>(w[q] >> 16);
    }
  }
}

template <int DT>
__device__ __forceinline__ u4 narrow(const float* v) {
  if constexpr (DT == ZERO_DT_F32)
    return (u4){__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  else
    return (u4){pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
}

template <typename T = u4>
__device__ __forceinline__ T load_any(const void* p) {
  T x;
  __builtin_memcpy(&x, p, sizeof x);
  return x;
}

// The same with the non-temporal hint: data that a pass touches once.
typedef u4 u4_any __attribute__((aligned(2)));
__device__ __forceinline__ u4 load_once(const void* p) { return __builtin_nontemporal_load(static_cast<const u4_any*>(p)); }
__device__ __forceinline__ void store_once(void* p, u4 x) { __builtin_nontemporal_store(x, static_cast<u4_any*>(p)); }

// The values at p, as far as `left` of them exist; the rest 0.
template <int DT, bool ONCE = false, typename Left>
__device__ __forceinline__ u4 load_part(const char* p, Left left) {
  if (left >= Vec<DT>::kVals) return ONCE ? load_once(p) : load_any(p);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int q = 0; q < Vec<DT>::kVals; ++q)
    if (q < left) {
      if constexpr (DT == ZERO_DT_F32) w[q] = reinterpret_cast<const uint32_t*>(p)[q];
      else w[q / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[q]) << (16 * (q & 1));
    }
  return (u4){w[0], w[1], w[2], w[3]};
}

// Values [first, end) of a slot at p.
template <int DT>
__device__ __forceinline__ void store_some(char* p, int first, int end, u4 x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int q = 0; q < Vec<DT>::kVals; ++q)
    if (q >= first && q < end) {
      if constexpr (DT == ZERO_DT_F32) reinterpret_cast<uint32_t*>(p)[q] = w[q];
      else reinterpret_cast<uint16_t*>(p)[q] = static_cast<uint16_t>(w[q / 2] >> (16 * (q & 1)));
    }
}

template <int DT, typename Left>
__device__ __forceinline__ void store_part(char* p, Left left, u4 x) {
  if (left >= Vec<DT>::kVals) store_once(p, x);
  else store_some<DT>(p, 0, static_cast<int>(left), x);
}

// One value of a type known at run time.
__device__ __forceinline__ float load_one(const void* p, int64_t i, int32_t dt) {
  if (dt == ZERO_DT_F32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dt == ZERO_DT_BF16 ? widen16<ZERO_DT_BF16>(h) : widen16<ZERO_DT_F16>(h);
}

__device__ __forceinline__ void store_one(void* p, int64_t i, int32_t dt, float v) {
  if (dt == ZERO_DT_F32) static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] =
        static_cast<uint16_t>(dt == ZERO_DT_BF16 ? pack2<ZERO_DT_BF16>(v, v) : pack2<ZERO_DT_F16>(v, v));
}

}  // namespace
}  // namespace zdp
