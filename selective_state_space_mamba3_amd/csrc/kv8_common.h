// Device helpers of the 8-bit key / value cache: a code is an OCP e4m3 number
// (largest 448, no infinity), its block's scale a power of two held as its
// exponent + 127.
#pragma once

#include "attn_common.h"
#include "kv8.h"

namespace m3 {

// A scale's exponent lies in [-110, 120]: the least code, 2^-119, is a normal number of bfloat16 and float32, and the
// largest that is written at 2^120 is 240, since 256 * 2^120 is more than either holds; so what a cache stands for is
// exact in both.  (Beyond 240 * 2^120 a value is off by at most the half step that any code may be, up to float32's end.)
constexpr int kExpBias = 127, kLeastExp = -110, kMostExp = 120;
constexpr float kLargestHeld = 0x1.ep127f;  // 240 * 2^120

// 2^e for e in -127 .. 127.
__device__ __forceinline__ float power_of_two(int e) { return __builtin_amdgcn_ldexpf(1.f, e); }
// The value of a scale byte.  (m3_kv8_write leaves 17 to 247; others are bent to 1 to 254, whose values are finite
// and not zero, so that a scale that goes with no token makes no NaN of a zero.)
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(min(max(byte, 1u), 254u) << 23); }
// The exponent that a block's older tokens have left it.
__device__ __forceinline__ int held_exponent(uint32_t byte) { return (int)min(byte, 254u) - kExpBias; }

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
// A number as the cache can hold it: nothing above kLargestHeld (no float16 is), NaN for what is not finite.
template <class T>
__device__ __forceinline__ float held(float x) {
  const float top = __is_same(T, _Float16) ? x : __builtin_amdgcn_fmed3f(x, -kLargestHeld, kLargestHeld);
  return __builtin_fabsf(x) < kInf ? top : __builtin_nanf("");
}
__device__ __forceinline__ floatx4 values4(uint32_t codes) {
  const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
  const floatx2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
  return floatx4{lo[0], lo[1], hi[0], hi[1]};
}

// Eight elements of a token, and eight codes, from column `col` (a multiple of 8); columns past D read as zero.
template <class T, bool VEC>
__device__ __forceinline__ Raw8<T> read_elements(const T* p, uint32_t col, uint32_t D) {
  Raw8<T> out;
  if constexpr (VEC) {
    out = *reinterpret_cast<const Raw8<T>*>(p + col);
  } else {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = col + i < D ? p[col + i] : (T)0.f;
    __builtin_memcpy(&out, e, sizeof out);
  }
  return out;
}
template <bool VEC>
__device__ __forceinline__ void write_codes(uint8_t* p, uint32_t col, uint32_t D, uintx2 c) {
  if constexpr (VEC) {
    *reinterpret_cast<uintx2*>(p + col) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < D) p[col + i] = (uint8_t)(c[i / 4] >> 8 * (i % 4));
  }
}
template <bool VEC>
__device__ __forceinline__ uintx2 read_codes(const uint8_t* p, uint32_t col, uint32_t D) {
  if constexpr (VEC) return *reinterpret_cast<const uintx2*>(p + col);
  uintx2 c = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + i < D) c[i / 4] |= (uint32_t)p[col + i] << 8 * (i % 4);
  return c;
}

// Eight elements times 2^-e (`inv`) as codes, and eight codes at another scale.
template <class T>
__device__ __forceinline__ uintx2 quantise8(const Raw8<T>& raw, float inv) {
  float f[8];
  raw_floats<T>(raw, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = held<T>(f[i]) * inv;
  return uintx2{codes4(f[0], f[1], f[2], f[3]), codes4(f[4], f[5], f[6], f[7])};
}
__device__ __forceinline__ uintx2 rescale8(uintx2 codes, float by) {
  const floatx4 lo = values4(codes[0]) * by, hi = values4(codes[1]) * by;
  return uintx2{codes4(lo[0], lo[1], lo[2], lo[3]), codes4(hi[0], hi[1], hi[2], hi[3])};
}
// The largest finite magnitude of eight elements and amax.  (Of their bits, 16-bit ones two at a time: a float maximum
// gives a signalling NaN in place of the number beside it, and the next one drops both.)
template <class T>
__device__ __forceinline__ float max_finite8(const Raw8<T>& raw, float amax) {
  if constexpr (sizeof(T) == 2) {
    typedef uint16_t ushortx2 __attribute__((ext_vector_type(2)));
    constexpr uint16_t inf = __is_same(T, _Float16) ? 0x7c00 : 0x7f80;
    ushortx2 top = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      top = __builtin_elementwise_max(top, __builtin_bit_cast(ushortx2, raw.v[0][i] & 0x7fff7fffu));
    uint16_t most = max(top[0], top[1]);
    // infinities and NaN are the largest
    if (__any(most >= inf)) {
      most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint16_t u = (uint16_t)(raw.v[0][i / 2] >> 16 * (i % 2)) & 0x7fff;
        most = max(most, u < inf ? u : (uint16_t)0);
      }
    }
    return __builtin_fmaxf(amax, to_float(__builtin_bit_cast(T, most)));
  } else {
    constexpr uint32_t inf = 0x7f800000u;
    float f[8];
    uint32_t u[8], most = 0;
    raw_floats<T>(raw, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u[i] = __float_as_uint(f[i]) & 0x7fffffffu;
      most = max(most, u[i]);
    }
    if (__any(most >= inf)) {
      most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) most = max(most, u[i] < inf ? u[i] : 0u);
    }
    return __builtin_fmaxf(amax, __uint_as_float(most));
  }
}

// Eight values from column `col` of a row, rounded once.
template <class T, bool VEC>
__device__ __forceinline__ void write_elements(T* p, uint32_t col, uint32_t D, const floatx4 f[2]) {
  if constexpr (VEC && sizeof(T) == 2) {
    *reinterpret_cast<uintx4*>(p + col) = uintx4{pack2<T>(f[0][0], f[0][1]), pack2<T>(f[0][2], f[0][3]),
                                                 pack2<T>(f[1][0], f[1][1]), pack2<T>(f[1][2], f[1][3])};
  } else if constexpr (VEC) {
    reinterpret_cast<floatx4*>(p + col)[0] = f[0];
    reinterpret_cast<floatx4*>(p + col)[1] = f[1];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < D) p[col + i] = (T)f[i / 4][i % 4];
  }
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
