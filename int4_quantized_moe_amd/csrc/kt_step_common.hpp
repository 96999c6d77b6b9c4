// Device helpers of the operators in kt_step.h.
#pragma once

#include "../../include/kt_step.h"
#include "kt_common.hpp"
#include "kt_internal.hpp"

namespace kt {

typedef uint32_t u32pair __attribute__((ext_vector_type(2)));

// Rows of 16 lanes exchanged between two registers: swap16 gives (a0, b0, a2, b2)
// and (a1, b1, a3, b3), swap32 (a0, a1, b0, b1) and (a2, a3, b2, b3), by rows.
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const u32pair r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r.x, b = r.y;
}
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const u32pair r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r.x, b = r.y;
}

// Two numbers rounded to nearest even, a in the low half, by one instruction; a NaN stays one.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 pair __attribute__((ext_vector_type(2)));
  const pair p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}

// The sum or maximum over a wave's lanes, the same bits in every lane.
__device__ __forceinline__ float rows_sum(float v) {
  uint32_t a = __float_as_uint(v), b = a;
  swap16(a, b);
  v = __uint_as_float(a) + __uint_as_float(b);
  a = b = __float_as_uint(v);
  swap32(a, b);
  return __uint_as_float(a) + __uint_as_float(b);
}
__device__ __forceinline__ float rows_max(float v) {
  uint32_t a = __float_as_uint(v), b = a;
  swap16(a, b);
  v = fmaxf(__uint_as_float(a), __uint_as_float(b));
  a = b = __float_as_uint(v);
  swap32(a, b);
  return fmaxf(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ float wave_sum(float v) { return rows_sum(row16_sum(v)); }
__device__ __forceinline__ float wave_max(float v) { return rows_max(row16_max(v)); }

}  // namespace kt
