// The 8-bit cache's element: an e4m3 code times a power of two kept per row
// (pa_cache.h). Conversions are the hardware's (cvt.rn to and from e4m3x2);
// the exponents are handled as bits.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace pa {

constexpr int kExpMin = -32;   // least exponent a row is held with
constexpr int kExpBias = 127;  // of the exponent byte

// The attention folds 2^e of a V row into its weight and takes it out of the sum again, a product
// of up to 2^31 keys' 2^-e. Bytes below this one (2^-64; writing a row makes none, a slot that was
// never written holds 0) count as it there: what they stand for, 448 * 2^-64 and less, is
// nothing beside fp16's least number, 2^-24, and sums of 2^64 stay far from fp32's end.
constexpr int kExpLeastByte = 63;

// e: the least integer >= kExpMin with a <= 448 * 2^e, a >= 0 finite.
// 448 = 1.75 * 2^8, so e = k - 8 for a = m * 2^k with m <= 1.75, else k - 7
// (zero and subnormal a have k = -127 here and end at kExpMin).
__device__ __forceinline__ int row_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int k = int(u >> 23) - 127;
  const int e = k - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kExpMin);
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Two values to e4m3 (lo in the low byte): nearest even, NaN for NaN, the
// largest finite code for an infinity.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp16 values to e4m3, likewise.
__device__ __forceinline__ uint32_t half2_e4m3x2(uint32_t a) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(a));
  return r;
}

// 2^e in both halves, e in [-14, 15].
__device__ __forceinline__ uint32_t half2_pow2(int e) {
  const uint32_t h = uint32_t(e + 15) << 10;
  return h | h << 16;
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The larger of each half; the other one's where one is NaN.
__device__ __forceinline__ uint32_t max_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two e4m3 codes (low 16 bits) to fp16, exact.
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(codes)));
  return r;
}

}  // namespace pa
