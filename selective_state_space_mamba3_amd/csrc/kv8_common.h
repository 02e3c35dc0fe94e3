// Device helpers of the 8-bit key / value cache: a code is an OCP e4m3 number
// (largest 448, no infinity), its block's scale a power of two held as its
// exponent + 127.
#pragma once

#include "attn_common.h"
#include "kv8.h"

namespace m3 {

// A scale's exponent lies in [-110, 120]: 448 * 2^120 holds every float32, and the least code, 2^-119, is a
// normal number of bfloat16 and float32, so that what a cache stands for is exact in both.
constexpr int kExpBias = 127, kLeastExp = -110, kMostExp = 120;

// 2^e for e in -126 .. 127.
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// The value of a scale byte.  (m3_kv8_write leaves 17 to 247; 0 counts as 1, so that a scale is never zero.)
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(max(byte, 1u) << 23); }

// The least exponent with amax <= 448 * 2^e (448 = 1.75 * 2^8; amax finite and not negative).
__device__ __forceinline__ int least_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kLeastExp), kMostExp);
}

// Four values as codes, to nearest with ties to even; what is not finite becomes NaN.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
__device__ __forceinline__ float finite_or_nan(float x) {
  return __builtin_fabsf(x) < kInf ? x : __builtin_nanf("");
}
__device__ __forceinline__ floatx4 values4(uint32_t codes) {
  const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
  const floatx2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
  return floatx4{lo[0], lo[1], hi[0], hi[1]};
}

// Page and row of a position of sequence b; page -1 where the table names none.
struct Slot {
  int page;
  uint32_t row;
};
__device__ __forceinline__ Slot find_slot(const int32_t* table, uint32_t b, uint32_t j, uint32_t page_size,
                                          uint32_t max_pages, uint32_t num_pages) {
  const uint32_t p = j / page_size;
  const int id = table == nullptr ? (int)b : table[(size_t)b * max_pages + p];
  return {id >= 0 && id < (int)num_pages ? id : -1, j - p * page_size};
}

}  // namespace m3
